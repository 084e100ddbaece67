"""Attention over the 8-bit key-value cache on the GPU against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

from oracle import kv_oracle as ko
from _kv import TYPES, Batch, assert_attention, attention_bound, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_int8_matmul_gb300 as q
    return q


def run(q, batch, kind, group, causal=True, scale=None, stride=0, max_tokens=None, extra=0, x=None, kernel=None):
    t, dim = TYPES[kind], batch.dim
    heads = batch.heads * group
    if x is None:
        x = rounded(batch.rng.standard_normal((batch.rows, heads, dim)) * 0.2, kind)
    big = torch.zeros((batch.rows + extra, heads + 1, dim + stride), dtype=t, device="cuda")
    big[:batch.rows, :heads, :dim] = torch.from_numpy(x).to(t).cuda()
    dq = big[:, :heads, :dim]
    cache, table, lengths, starts = batch.device(q)
    out = torch.full((batch.rows + extra, heads, dim), 7.0, dtype=t, device="cuda")
    y = q.qmm_kv_attention(dq, cache, table, lengths, starts=starts, scale=scale, causal=causal, max_tokens=max_tokens,
                           out=out)
    assert y.data_ptr() == out.data_ptr()
    if kernel:
        assert q.last_kernel() == kernel
    s = dim ** -0.5 if scale is None else scale
    exact, mag, top, seen = ko.attention(x.astype(np.float64), *batch.cache_arrays(), batch.table, batch.lengths,
                                         batch.starts, s, causal, detail=True)
    got = y.double().cpu().numpy()
    assert (got[batch.rows:] == 7).all()
    assert_attention(got[:batch.rows], exact, attention_bound(exact, mag, top, seen, kind, dim))
    q.check_device_error()
    return y


ODD = [(1, 1), (1, 0), (0, 30), (2, 17), (1, 16), (1, 15), (3, 2), (4, 100), (1, 333), (7, 64)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page,heads,group", [(64, 16, 1, 1), (128, 64, 2, 4), (64, 48, 3, 3), (128, 16, 1, 8),
                                                  (128, 32, 2, 16), (64, 64, 5, 7), (128, 48, 1, 20)])
@pytest.mark.parametrize("causal", [True, False])
def test_sequences_of_all_kinds(q, kind, dim, page, heads, group, causal):
    run(q, Batch(ODD, heads, dim, page, seed=group), kind, group, causal, extra=3)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_single_tokens(q, kind):
    for dim, group in ((128, 4), (64, 2)):
        run(q, Batch([(1, n) for n in (1, 2, 16, 31, 64, 65, 500, 1021)], 2, dim, 64, starts=False), kind, group,
            max_tokens=1)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim,heads,group", [(128, 1, 8), (64, 8, 1)])
def test_one_long_sequence_is_split(q, kind, dim, heads, group):
    run(q, Batch([(1, 9000)], heads, dim, 64), kind, group)
    run(q, Batch([(1, 7001), (1, 3), (2, 1100)], heads, dim, 16), kind, group)


@pytest.mark.parametrize("stride", [1, 8])
def test_strided_queries(q, stride):
    for kind in ("bf16", "f32"):
        run(q, Batch(ODD, 2, 64, 16, seed=1), kind, 2, stride=stride)


def test_bad_pages_and_short_tables_are_not_seen(q):
    seqs = [(1, 100), (3, 64), (2, 33), (1, 17), (1, 16)]
    for kind in ("bf16", "f32"):
        run(q, Batch(seqs, 2, 64, 16, bad=((0, 0, -1), (0, 3, 1 << 30), (2, 1, 500), (4, 0, -5))), kind, 2)
        run(q, Batch(seqs, 2, 128, 16, width=2), kind, 3)
        run(q, Batch(seqs, 2, 64, 16, width=0), kind, 2)


def test_scales_far_apart_in_a_sequence(q):
    """Blocks whose powers of two differ by up to 2^40, the large ones first, last and between."""
    for kind in ("bf16", "f32"):
        for order in (1, -1):
            b = Batch([(1, 200), (2, 90)], 2, 64, 16, seed=4)
            b.ve[:] = np.linspace(100, 140, b.ve.size).astype(np.uint8).reshape(b.ve.shape)[::order]
            run(q, b, kind, 2)
        b = Batch([(1, 200)], 2, 64, 16, seed=4)
        b.ke[:] = b.rng.integers(100, 122, b.ke.shape)
        run(q, b, kind, 2)


def test_queries_of_all_magnitudes(q):
    for kind in ("bf16", "f32"):
        b = Batch([(6, 200)], 1, 64, 16, seed=5)
        x = rounded(b.rng.standard_normal((6, 2, 64)) * np.array([1e-38, 1e-20, 1e-3, 1, 3, 0])[:, None, None], kind)
        run(q, b, kind, 2, x=x)


def test_rows_that_are_not_finite(q):
    for kind in ("bf16", "f32"):
        b = Batch([(4, 200)], 2, 64, 16, seed=6)
        x = rounded(b.rng.standard_normal((4, 4, 64)) * 0.2, kind)
        x[0, 0, 5], x[1, 3, 0], x[3, 1, 63] = np.nan, np.inf, -np.inf
        cache, table, lengths, starts = b.device(q)
        y = q.qmm_kv_attention(torch.from_numpy(x).to(TYPES[kind]).cuda(), cache, table, lengths, starts)
        y = y.double().cpu().numpy()
        bad = np.zeros((4, 4), bool)
        bad[0, 0] = bad[1, 3] = bad[3, 1] = True
        assert np.isnan(y[bad]).all()
        x[bad] = 0
        exact, mag, top, seen = ko.attention(x.astype(np.float64), *b.cache_arrays(), b.table, b.lengths, b.starts,
                                             64 ** -0.5, True, detail=True)
        bound = attention_bound(exact, mag, top, seen, kind, 64)
        assert_attention(y[~bad], exact[~bad], bound[~bad])


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_other_scales(q, scale):
    for kind in ("bf16", "f32"):
        run(q, Batch(ODD, 2, 64, 16, seed=7), kind, 2, scale=scale)


def test_same_call_same_bits(q):
    b = Batch([(1, 3000), (3, 500)], 2, 128, 64, seed=8)
    x = rounded(b.rng.standard_normal((4, 8, 128)), "bf16")
    args = b.device(q)
    d = torch.from_numpy(x).bfloat16().cuda()
    first = q.qmm_kv_attention(d, *args)
    for _ in range(3):
        assert torch.equal(first, q.qmm_kv_attention(d, *args))


@pytest.mark.parametrize("dim,page,heads,group", [(64, 16, 2, 1), (128, 64, 1, 4), (64, 48, 1, 3), (128, 16, 2, 8),
                                                  (128, 128, 1, 1)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_prompts(q, kind, dim, page, heads, group, causal):
    """Sequences of many rows, alone and among short ones; ends inside tiles of rows and of tokens."""
    for seqs in ([(200, 200)], [(17, 17), (129, 300), (1, 400), (0, 3), (64, 64), (2, 1), (70, 40)],
                 [(128, 128), (128, 257)]):
        run(q, Batch(seqs, heads, dim, page, seed=dim), kind, group, causal)


def test_prompts_of_equal_length_take_one_kernel(q):
    for kind, few in (("bf16", 4), ("f32", 8)):
        run(q, Batch([(40, 300), (40, 40), (40, 39)], 2, 64, 16), kind, 4, max_tokens=40, kernel="kv_attention_tiles")
        run(q, Batch([(40, 300), (3, 40)], 2, 64, 16), kind, 4, max_tokens=40, kernel="kv_attention_rows+tiles")
        run(q, Batch([(few, 300), (3, 40)], 2, 64, 16), kind, 4, max_tokens=few, kernel="kv_attention_rows")


def test_a_wrong_hint_costs_time_only(q):
    for kind in ("bf16", "f32"):
        for hint in (1, 3, 1000):
            run(q, Batch([(40, 300), (3, 40), (17, 60)], 2, 128, 16), kind, 4, max_tokens=hint)


def test_prompt_pieces_are_split_over_tokens(q):
    """Few items, many tokens: parts of one item from several CTAs."""
    for kind in ("bf16", "f32"):
        run(q, Batch([(33, 6000)], 1, 128, 64, seed=3), kind, 4)
        run(q, Batch([(20, 3000), (5, 9)], 1, 64, 16, seed=3), kind, 8)


def test_prompts_with_bad_pages_and_short_tables(q):
    seqs = [(40, 100), (30, 300), (33, 33)]
    bad = ((0, 0, -1), (0, 3, 1 << 30), (1, 1, 500), (1, 8, -2), (2, 0, -5))
    for kind in ("bf16", "f32"):
        run(q, Batch(seqs, 2, 64, 16, bad=bad), kind, 2)
        run(q, Batch(seqs, 2, 128, 16, width=7), kind, 3)
        run(q, Batch(seqs, 2, 64, 48, width=0), kind, 2)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_prompt_scales_queries_and_strides(q, kind):
    for order in (1, -1):
        b = Batch([(40, 700), (20, 90)], 2, 64, 16, seed=4)
        b.ve[:] = np.linspace(100, 140, b.ve.size).astype(np.uint8).reshape(b.ve.shape)[::order]
        b.ke[:] = b.rng.integers(100, 122, b.ke.shape)
        run(q, b, kind, 2, stride=1)
    b = Batch([(24, 200)], 1, 128, 16, seed=5)
    mags = np.resize([1e-38, 1e-20, 1e-3, 1, 3, 0], 24)[:, None, None]
    run(q, b, kind, 2, x=rounded(b.rng.standard_normal((24, 2, 128)) * mags, kind), stride=8, extra=5)
    run(q, Batch([(50, 200)], 1, 128, 16, seed=5), kind, 2, stride=1)
    for scale in (0.0, -0.3, 2.0):
        run(q, Batch([(40, 150), (18, 17)], 2, 64, 16, seed=7), kind, 2, scale=scale)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_prompt_rows_that_are_not_finite(q, kind):
    b = Batch([(40, 200)], 1, 64, 16, seed=6)
    x = rounded(b.rng.standard_normal((40, 4, 64)) * 0.2, kind)
    bad = np.zeros((40, 4), bool)
    for i, (t, h) in enumerate(((0, 0), (17, 3), (39, 1))):
        x[t, h, 5 * i], bad[t, h] = (np.nan, np.inf, -np.inf)[i], True
    cache, table, lengths, starts = b.device(q)
    y = q.qmm_kv_attention(torch.from_numpy(x).to(TYPES[kind]).cuda(), cache, table, lengths, starts).double().cpu().numpy()
    assert np.isnan(y[bad]).all()
    x[bad] = 0
    exact, mag, top, seen = ko.attention(x.astype(np.float64), *b.cache_arrays(), b.table, b.lengths, b.starts,
                                         64 ** -0.5, True, detail=True)
    bound = attention_bound(exact, mag, top, seen, kind, 64)
    assert_attention(y[~bad], exact[~bad], bound[~bad])
