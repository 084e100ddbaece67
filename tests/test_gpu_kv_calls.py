"""The key-value cache's calls as a server makes them: on streams, captured and replayed, two
at once, next to memory that is not theirs, and far into large caches."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as ko
from _kv import TYPES, Batch, assert_attention, attention_bound, rounded, turns
from test_gpu_layer_guards import Guards

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")

MIXED = [(1, 1), (3, 40), (0, 20), (60, 60), (17, 130), (1, 333)]


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check(b, x, y, kind="bf16", causal=True):
    exact, mag, top, seen = ko.attention(x.astype(np.float64), *b.cache_arrays(), b.table, b.lengths, b.starts,
                                         b.dim ** -0.5, causal, detail=True)
    assert_attention(y.double().cpu().numpy(), exact, attention_bound(exact, mag, top, seen, kind, b.dim))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 48)])
def test_nothing_is_written_outside(kind, dim, page):
    """Outputs, workspace and cache between guard bytes; rows behind the last sequence's stay as they are, and so do
    pages that no row of the table names."""
    t, b = TYPES[kind], Batch(MIXED, 2, dim, page, seed=1, spare=5)
    rows, extra, heads = b.rows, 4, 6
    g = Guards()
    cache = q.KvCache(*(g(a.shape, torch.from_numpy(a).dtype) for a in b.cache_arrays()))
    for c, a in zip(cache, b.cache_arrays()):
        c.copy_(torch.from_numpy(a))
    _, table, lengths, starts = b.device(q)
    gen = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(rows + extra, 2, dim, generator=gen, device="cuda").to(t) for _ in range(2))
    x = torch.randn(rows + extra, heads, dim, generator=gen, device="cuda").to(t)
    cos, sin = (torch.from_numpy(a).cuda() for a in turns(400, dim // 2))
    qo, out, ko_, vo = (g(s, t) for s in ((rows + extra, heads, dim),) * 2 + ((rows + extra, 2, dim),) * 2)
    for o in (qo, out, ko_, vo):
        o.fill_(7)
    ws = g((q.qmm_kv_attention_workspace_bytes(rows + extra, len(MIXED), heads, 2, dim, t),), torch.uint8)
    used = set(b.table[b.table >= 0].tolist())
    q.qmm_kv_append(cache, k, v, table, lengths, starts=starts, q=x, cos=cos, sin=sin, q_out=qo)
    q.qmm_kv_read(cache, table, lengths, starts, rows=rows + extra, k_out=ko_, v_out=vo)
    q.qmm_kv_attention(qo, cache, table, lengths, starts=starts, out=out, workspace=ws)
    g.check()
    q.check_device_error()
    for o in (qo, out, ko_, vo):
        assert (o[rows:] == 7).all() and not (o[:rows] == 7).all()
    for c, a in zip(cache, b.cache_arrays()):
        c = c.cpu().numpy()
        for p in set(range(b.pages)) - used:
            assert np.array_equal(c[p], a[p])


def test_given_streams_own_what_the_calls_allocate():
    from test_gpu_given_stream import check_owner
    b = Batch(MIXED, 2, 64, 16, seed=3)
    cache, table, lengths, starts = b.device(q)
    k, v = (torch.randn(b.rows, 2, 64, device="cuda").bfloat16() for _ in range(2))
    x = torch.randn(b.rows, 6, 64, device="cuda").bfloat16()
    check_owner(lambda s: (q.qmm_kv_append(cache, k, v, table, lengths, starts=starts, q=x, stream=s),))
    check_owner(lambda s: q.qmm_kv_read(cache, table, lengths, starts, rows=b.rows, stream=s))
    check_owner(lambda s: (q.qmm_kv_attention(x, cache, table, lengths, starts=starts, stream=s),))
    few = Batch([(1, n) for n in (5, 700, 33)], 2, 64, 16, seed=3, starts=False)
    cache, table, lengths, _ = few.device(q)
    check_owner(lambda s: (q.qmm_kv_attention(x[:3], cache, table, lengths, stream=s),))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_a_captured_step_follows_lengths_and_tables(kind):
    """One captured append and attention, replayed as the sequences grow, change pages and end."""
    t = TYPES[kind]
    b = Batch([(1, 1)] * 3, 2, 64, 16, width=8, spare=30, starts=False)
    b.table[:] = b.rng.permutation(24).reshape(3, 8)
    cache, table, lengths, _ = b.device(q)
    arrays = b.cache_arrays()
    cos, sin = turns(128, 32)
    dc, ds = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
    x = torch.zeros(3, 8, 64, dtype=t, device="cuda")     # 4 query, 2 key, 2 value heads
    out = torch.empty(3, 4, 64, dtype=t, device="cuda")

    def step():
        r = q.qmm_kv_append(cache, x[:, 4:6], x[:, 6:], table, lengths, q=x[:, :4], cos=dc, sin=ds)
        q.qmm_kv_attention(r, cache, table, lengths, out=out, max_tokens=1)
        return r

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lengths.zero_()                                    # warm-up that stores nothing
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turned = step()
    for i in range(40):
        n = np.array([i + 1, min(2 * i + 1, 128), 60 - i if i < 3 else 0], np.int32)
        if i == 20:
            b.table[:] = b.table[:, ::-1]                  # other pages from here on: what they hold is history
            table.copy_(torch.from_numpy(b.table.copy()))
        new = rounded(b.rng.standard_normal((3, 8, 64)), kind)
        x.copy_(torch.from_numpy(new))
        lengths.copy_(torch.from_numpy(n))
        graph.replay()
        want = ko.append(*arrays, new[:, 4:6], new[:, 6:], b.table, n, None, cos, sin, False, new[:, :4])
        for got, w in zip(cache, arrays):
            assert np.array_equal(got.cpu().numpy(), w), i
        assert np.array_equal(turned.float().cpu().numpy(), rounded(want, kind), equal_nan=True)
        xq = turned.double().cpu().numpy()
        xq[np.isnan(xq).any(axis=(1, 2))] = 0              # (a sequence without tokens: its position has no rotation)
        exact, mag, top, seen = ko.attention(xq, *arrays, b.table, n, None, 64 ** -0.5, True, detail=True)
        got = out.double().cpu().numpy()
        ended = n == 0
        assert_attention(got[~ended], exact[~ended], attention_bound(exact, mag, top, seen, kind, 64)[~ended], i)


def test_two_prompts_at_once_on_two_streams():
    b = [Batch([(150, 400), (1, 900)], 2, 64, 16, seed=i) for i in (1, 2)]
    xs = [rounded(c.rng.standard_normal((c.rows, 8, 64)), "bf16") for c in b]
    args = [(torch.from_numpy(x).bfloat16().cuda(), *c.device(q)) for x, c in zip(xs, b)]
    streams = [torch.cuda.Stream() for _ in b]
    torch.cuda.synchronize()
    for _ in range(5):
        ys = [q.qmm_kv_attention(*a[:4], starts=a[4], stream=s) for a, s in zip(args, streams)]
    torch.cuda.synchronize()
    for c, x, y in zip(b, xs, ys):
        check(c, x, y)
    q.check_device_error()


def test_one_workspace_for_calls_in_turn():
    """Calls of several shapes with one workspace, in stream order, and what is left in it before."""
    ws = torch.full((q.qmm_kv_attention_workspace_bytes(200, 8, 16, 1, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    for seqs, group in (([(100, 500)], 4), ([(1, 3000)], 8), ([(150, 150), (2, 9)], 3), ([(1, 1)], 1)):
        b = Batch(seqs, 1, 128, 16, seed=group)
        x = rounded(b.rng.standard_normal((b.rows, group, 128)), "bf16")
        d = torch.from_numpy(x).bfloat16().cuda()
        a = b.device(q)
        check(b, x, q.qmm_kv_attention(d, *a, workspace=ws))
        need = q.qmm_kv_attention_workspace_bytes(b.rows, len(seqs), group, 1, 128)
        with pytest.raises(q.QmmError):
            q.qmm_kv_attention(d, *a, workspace=ws[:need - 1])


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: pages at its end, for both kernels, appended to, read and attended to."""
    pages, heads, dim, page = 2 ** 32 // (8 * 128 * 64) + 70, 8, 128, 64
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("memory")
    cache = q.KvCache(*(torch.empty(pages, heads, page, dim, dtype=torch.int8, device="cuda") for _ in range(2)),
                      *(torch.empty(pages, heads, page // 16, dtype=torch.uint8, device="cuda") for _ in range(2)))
    small = q.qmm_kv_cache(3, heads, dim, page=page)
    far = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(150, heads, dim, device="cuda").bfloat16() for _ in range(2))
    x = torch.randn(150, 16, dim, device="cuda").bfloat16()
    outs = []
    for c, table in ((cache, far), (small, near)):
        q.qmm_kv_append(c, k, v, table, ints(150), starts=ints(0, 150))
        outs.append([*q.qmm_kv_read(c, table, ints(150), ints(0, 150), rows=150),
                     q.qmm_kv_attention(x, c, table, ints(150), starts=ints(0, 150)),
                     q.qmm_kv_attention(x[:1], c, table, ints(150))])
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    q.check_device_error()


def test_large_strides():
    """Rows more than 2^31 elements apart."""
    step = 2 ** 31 // 3 + 64
    if torch.cuda.mem_get_info()[0] < 24 * 2 ** 30:
        pytest.skip("memory")
    big = torch.empty(4 * step, dtype=torch.bfloat16, device="cuda")
    b = Batch([(4, 100)], 1, 64, 16, seed=4)
    cache, table, lengths, starts = b.device(q)
    x = rounded(b.rng.standard_normal((4, 4, 64)), "bf16")
    view = big.as_strided((4, 4, 64), (step, 64, 1))
    view.copy_(torch.from_numpy(x))
    check(b, x, q.qmm_kv_attention(view, cache, table, lengths, starts=starts, max_tokens=1))
    check(b, x, q.qmm_kv_attention(view, cache, table, lengths, starts=starts, max_tokens=4))
    arrays = b.cache_arrays()
    r = q.qmm_kv_append(cache, view[:, 1:2], view[:, 2:3], table, lengths, starts=starts, q=view)
    ko.append(*arrays, x[:, 1:2], x[:, 2:3], b.table, b.lengths, b.starts)
    for got, w in zip(cache, arrays):
        assert np.array_equal(got.cpu().numpy(), w)
    assert np.array_equal(r.float().cpu().numpy(), x)


def test_in_place_rotation():
    b = Batch([(5, 30)], 2, 64, 16, seed=5)
    cos, sin = turns(40, 32)
    x = torch.randn(5, 3, 64, device="cuda").bfloat16()
    k = torch.randn(5, 2, 64, device="cuda").bfloat16()
    args = dict(cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda())
    cache, table, lengths, starts = b.device(q)
    want = q.qmm_kv_append(cache, k, k, table, lengths, starts=starts, q=x, **args)
    got = q.qmm_kv_append(cache, k, k, table, lengths, starts=starts, q=x, q_out=x, **args)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)


def test_pages_shared_by_sequences():
    """A common beginning on the same pages, the same page twice in a row: reading is free."""
    b = Batch([(1, 48), (20, 48), (1, 32)], 2, 64, 16, seed=6)
    b.table[1, :2] = b.table[0, :2]
    b.table[2, 1] = b.table[2, 0]
    x = rounded(b.rng.standard_normal((b.rows, 4, 64)), "bf16")
    d = torch.from_numpy(x).bfloat16().cuda()
    check(b, x, q.qmm_kv_attention(d, *b.device(q)))


def test_empty_calls():
    cache = q.qmm_kv_cache(2, 2, 64, page=16)
    none, table = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 4, 64, device="cuda")
    assert q.qmm_kv_append(cache, x[:, :2], x[:, :2], table, none, q=x).shape == x.shape
    assert q.qmm_kv_attention(x, cache, table, none).shape == x.shape
    assert q.qmm_kv_read(cache, table, none)[0].shape == (0, 2, 64)
    assert q.qmm_kv_attention(x, cache, torch.zeros(2, 3, dtype=torch.int32, device="cuda"), ints(5, 6),
                              starts=ints(0, 0, 0)).shape == x.shape
    # a cache without pages: nothing is there
    empty = q.qmm_kv_cache(0, 2, 64, page=16)
    y = q.qmm_kv_attention(torch.ones(40, 4, 64, device="cuda").bfloat16(), empty, ints(0, 1).view(1, 2), ints(30),
                           starts=ints(0, 40))
    assert not y.any()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_sequences_that_make_no_sense_touch_nothing_else(kind):
    """Starts out of order, negative or past the rows, lengths from -5 to 2^31 - 1: what comes out of them is not
    defined, but nothing outside the outputs, the workspace and the named pages is written."""
    t, heads, dim, page = TYPES[kind], 2, 64, 16
    b = Batch([(9, 40)] * 5, heads, dim, page, seed=9, spare=6)
    g = Guards()
    cache = q.KvCache(*(g(a.shape, torch.from_numpy(a).dtype) for a in b.cache_arrays()))
    for c, a in zip(cache, b.cache_arrays()):
        c.copy_(torch.from_numpy(a))
    table = torch.from_numpy(b.table).cuda()
    rows = 45
    x, k, v = (torch.randn(rows, h, dim, device="cuda").to(t) for h in (8, 2, 2))
    cos, sin = (torch.from_numpy(a).cuda() for a in turns(64, 32))
    used = set(b.table[b.table >= 0].tolist())
    for starts in ([5, 2, 100, -3, 7, 45], [0, 2 ** 31 - 1, -2 ** 31, 30, 3, 1], [45, 0, 45, 0, 45, 0]):
        for lengths in ([2 ** 31 - 1, -5, 40, 7, 0], [-2 ** 31, 1, 2 ** 30, 48, 49]):
            for most in (1, 9, 45):
                qo, out, kr, vr = (g((rows, h, dim), t) for h in (8, 8, 2, 2))
                ws = g((q.qmm_kv_attention_workspace_bytes(rows, 5, 8, heads, dim, t, most),), torch.uint8)
                s, n = ints(*starts), ints(*lengths)
                q.qmm_kv_append(cache, k, v, table, n, starts=s, q=x, cos=cos, sin=sin, q_out=qo)
                q.qmm_kv_read(cache, table, n, s, rows=rows, k_out=kr, v_out=vr)
                for causal in (True, False):
                    q.qmm_kv_attention(x, cache, table, n, starts=s, out=out, workspace=ws, causal=causal, max_tokens=most)
    g.check()
    q.check_device_error()
    for c, a in zip(cache, b.cache_arrays()):
        c = c.cpu().numpy()
        for p in set(range(b.pages)) - used:
            assert np.array_equal(c[p], a[p])
    good = Batch([(1, 30), (40, 70)], heads, dim, page, seed=10)
    y = rounded(good.rng.standard_normal((41, 4, dim)), kind)
    check(good, y, q.qmm_kv_attention(torch.from_numpy(y).to(t).cuda(), *good.device(q)), kind)
