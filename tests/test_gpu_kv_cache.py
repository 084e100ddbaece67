"""The 8-bit key-value cache on the GPU: appended blocks, rotated queries and tokens read
back, bit for bit against the plain form."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as ko
from _kv import TYPES, Batch, rounded, turns

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_int8_matmul_gb300 as q
    return q


def run_append(q, batch, kind, q_heads=4, half=0, interleaved=False, scale=1.0, stride=0, positions=None, tweak=None):
    rng, t = batch.rng, TYPES[kind]
    cos = sin = None
    if half:
        need = max([length for _, length in batch.seqs] + [1])
        cos, sin = turns(need if positions is None else positions, half)
    x = rounded(rng.standard_normal((batch.rows, q_heads + 2 * batch.heads, batch.dim)) * scale, kind)
    if tweak:
        tweak(x)
    hs = batch.heads
    # heads and rows further apart than they need be; stride odd: off 16 bytes
    big = torch.zeros((batch.rows, q_heads + 2 * hs, batch.dim + stride), dtype=t, device="cuda")
    big[..., :batch.dim] = torch.from_numpy(x).to(t).cuda()
    dq, dk, dv = (big[:, a:b, :batch.dim] for a, b in ((0, q_heads), (q_heads, q_heads + hs),
                                                       (q_heads + hs, q_heads + 2 * hs)))
    cache, table, lengths, starts = batch.device(q)
    dcos, dsin = (None, None) if cos is None else (torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda())
    got = q.qmm_kv_append(cache, dk, dv, table, lengths, starts=starts, q=dq, cos=dcos, sin=dsin,
                          interleaved=interleaved)
    arrays = batch.cache_arrays()
    want = ko.append(*arrays, x[:, q_heads:q_heads + hs], x[:, q_heads + hs:], batch.table, batch.lengths, batch.starts,
                     cos, sin, interleaved, x[:, :q_heads])
    assert q.last_kernel() == "kv_append"
    for name, g, w in zip(("k", "v", "k_exp", "v_exp"), cache, arrays):
        g = g.cpu().numpy()
        assert np.array_equal(g, w), (name, np.argwhere(g != w)[:5])
    assert np.array_equal(got.float().cpu().numpy(), rounded(want, kind), equal_nan=True)
    return cache, table, lengths, starts, (dq, dk, dv, dcos, dsin)


MIXED = [(1, 1), (1, 17), (0, 40), (5, 5), (16, 33), (33, 70), (1, 16), (3, 48)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, 1), (128, 64, 3), (64, 48, 9), (128, 16, 8)])
def test_append_is_the_definition_bit_for_bit(q, kind, dim, page, heads):
    run_append(q, Batch(MIXED, heads, dim, page, seed=dim + page), kind, q_heads=2 * heads, half=dim // 2)


@pytest.mark.parametrize("half,interleaved", [(8, False), (8, True), (16, True), (24, False), (32, True), (32, False),
                                              (0, False)])
@pytest.mark.parametrize("stride", [0, 8, 1])
def test_rotations_and_strides(q, half, interleaved, stride):
    run_append(q, Batch(MIXED, 2, 64, 32, seed=half), "bf16", q_heads=17, half=half, interleaved=interleaved,
               stride=stride)
    run_append(q, Batch(MIXED, 2, 128, 32, seed=half), "f32", q_heads=3, half=half, interleaved=interleaved,
               stride=stride)


def test_one_row_a_sequence_without_starts(q):
    run_append(q, Batch([(1, n) for n in range(1, 70)], 2, 64, 16, starts=False), "bf16", half=32)


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-3, 1.0, 1e4, 1e30, 1e38])
def test_scales_follow_the_numbers(q, scale):
    """Fresh blocks, blocks whose scale grows by a little and by everything, and ones that keep theirs."""
    for kind in ("bf16", "f32"):
        run_append(q, Batch(MIXED, 2, 64, 16, seed=3), kind, scale=scale)


def test_values_at_the_edge_of_a_scale(q):
    """Largest magnitudes of 127.5 steps and next to it; ties of every size; zeros."""
    def edge(x):
        flat = x[:, 4:].reshape(-1)
        flat[:] = np.resize(np.arange(-255, 256) / 2.0, flat.shape) * 2.0 ** -3
        x[0], x[1, :, 0] = 0.0, 127.5
        x[2, :, :] = np.float32(127.49999)
    for page in (16, 32):
        run_append(q, Batch(MIXED, 2, 64, page, seed=5), "f32", tweak=edge)


def test_not_finite_numbers(q):
    def spoil(x):
        x[0, :, 3], x[1, :, 1], x[2, :, 9], x[5, 0] = np.nan, np.inf, -np.inf, np.nan
    for half in (0, 32):
        run_append(q, Batch(MIXED, 2, 64, 16, seed=6), "bf16", half=half, tweak=spoil)


def test_tokens_without_a_place(q):
    """Negative positions, table rows that end, pages that do not exist, positions without a rotation."""
    seqs = [(9, 4), (20, 40), (4, 64), (3, 0), (2, 30), (40, 60)]
    run_append(q, Batch(seqs, 2, 64, 16, width=3, bad=((1, 1, -1), (4, 1, 99), (5, 2, 2 ** 31 - 1))), "bf16", half=32,
               positions=50)
    run_append(q, Batch(seqs, 2, 64, 16, width=0), "f32", half=16)


def test_many_sequences(q):
    rng = np.random.default_rng(9)
    seqs = []
    for _ in range(150):
        n = int(rng.integers(0, 20))
        seqs.append((n, n + int(rng.integers(0, 50))))
    run_append(q, Batch(seqs, 1, 64, 16, seed=8), "bf16", q_heads=2, half=32)


def test_appending_token_by_token(q):
    """Growth after growth: every token within one final step of itself, and what the plain form holds."""
    batch = Batch([(1, 1), (1, 1)], 2, 64, 16, spare=6, width=3)
    batch.table[:] = np.arange(6).reshape(2, 3)
    cache, table, _, _ = batch.device(q)
    arrays = batch.cache_arrays()
    rng = np.random.default_rng(1)
    ks = rounded(rng.standard_normal((40, 2, 2, 64)) * 1.3 ** np.arange(40)[:, None, None, None], "bf16")
    for i in range(40):
        lengths = np.full(2, i + 1, np.int32)
        d = torch.from_numpy(ks[i]).bfloat16().cuda()
        q.qmm_kv_append(cache, d, -d, table, torch.from_numpy(lengths).cuda())
        ko.append(*arrays, ks[i], -ks[i], batch.table, lengths, None)
    for g, w in zip(cache, arrays):
        assert np.array_equal(g.cpu().numpy(), w)
    k, v = q.qmm_kv_read(cache, table, torch.full((2,), 40, dtype=torch.int32, device="cuda"),
                         starts=torch.tensor([0, 40, 80], dtype=torch.int32, device="cuda"), rows=80,
                         out_dtype=torch.float32)
    got = k.cpu().numpy().reshape(2, 40, 2, 64)
    steps = ko.power(arrays[2][batch.table])                          # [sequence, page, head, 1]
    step = np.repeat(steps[..., 0].transpose(0, 1, 2), 16, axis=1)[:, :40]
    assert (np.abs(got - ks.transpose(1, 0, 2, 3)) <= step[..., None]).all()
    assert torch.equal(k, -v)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, 5), (128, 48, 3)])
def test_read_back(q, kind, dim, page, heads):
    seqs = [(9, 4), (0, 5), (1, 1), (20, 40), (33, 70)]
    b = Batch(seqs, heads, dim, page, seed=2, bad=((3, 0, -7),))
    cache, table, lengths, starts = b.device(q)
    out = torch.full((b.rows + 3, heads, dim), 7.0, dtype=TYPES[kind], device="cuda")
    k, v = q.qmm_kv_read(cache, table, lengths, starts, rows=b.rows + 3, k_out=out, v_out=out.clone(),
                         out_dtype=TYPES[kind])
    for got, c, e in ((k, b.kc, b.ke), (v, b.vc, b.ve)):
        want = ko.read(c, e, b.table, b.lengths, b.starts, b.rows)
        assert np.array_equal(got[:b.rows].double().cpu().numpy(), want)   # int8 * 2^n is exact in both types
        assert (got[b.rows:] == 7).all()                                   # rows behind the last sequence
    assert q.last_kernel() == "kv_read"


def test_read_of_the_smallest_steps(q):
    b = Batch([(3, 3)], 1, 64, 16)
    b.ke[:], b.ve[:] = 0, 1
    cache, table, lengths, starts = b.device(q)
    k, v = q.qmm_kv_read(cache, table, lengths, starts, rows=3, out_dtype=torch.float32)
    assert np.array_equal(k.double().cpu().numpy(), ko.read(b.kc, b.ke, b.table, b.lengths, b.starts, 3))
    assert np.array_equal(v.double().cpu().numpy(), ko.read(b.vc, b.ve, b.table, b.lengths, b.starts, 3))
