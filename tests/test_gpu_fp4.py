"""4-bit floats with block scales against the oracle: what is packed reads back bit
for bit (rows, columns, both; every tile edge, strides, types, non-finite blocks),
and products lie within the bound of one fp32 accumulation over K, from one row to
several tiles, at ragged sizes, for both blocks and outputs."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as O
from _helpers import half_ulp

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def f32(t):
    return t.float().cpu().numpy()


def make(R, C, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(R, C, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-6, 7, (R, 1), generator=g, device="cuda").float())
    return (x * torch.where(torch.rand(R, C, generator=g, device="cuda") < 0.01, 20.0, 1.0)).to(dt)


def check_values(m, x, bf16_out=False):
    want = O.fp4_values(f32(x), m.block, bf16_out)
    got = q.qmm_fp4_dequantize(m, out_dtype=torch.bfloat16 if bf16_out else torch.float32)
    got = f32(got)
    assert got.shape == want.shape
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    assert same.all(), f"{(~same).sum()} of {want.size} values differ, first at {np.argwhere(~same)[0]}"


SHAPES = [(1, 1), (1, 16), (2, 31), (3, 33), (1, 4096), (16, 8192), (127, 128), (128, 129), (129, 127), (130, 257),
          (64, 100), (300, 1000), (33, 4100), (257, 515), (5, 20000), (1, 70000), (1024, 200), (1025, 200),
          (200, 1024), (201, 1027), (2, 200001), (1100, 2055)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", SHAPES)
def test_quantise_reads_back(R, C, dt, block):
    x = make(R, C, TYPES[dt], R + 10 * C)
    rows = q.qmm_fp4_quantize(x, block=block)
    assert q.last_kernel().startswith("fp4_quantize_rows")
    assert (rows.rows, rows.cols, rows.block) == (R, C, block)
    check_values(rows, x)
    check_values(rows, x, True)
    xt = x.T.contiguous()
    cols = q.qmm_fp4_quantize(x, block=block, transpose=True)
    assert (cols.rows, cols.cols) == (C, R)
    check_values(cols, xt)
    check_values(q.qmm_fp4_quantize(xt, block=block, transpose=True), x)
    a, b = q.qmm_fp4_quantize_both(x, block=block)
    check_values(a, x)
    check_values(b, xt)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("ld,off", [(304, 0), (301, 0), (320, 1), (4096, 3)])
def test_quantise_strides_and_alignment(dt, block, ld, off):
    x = make(141, ld + off, TYPES[dt], 7)[:, off:off + 300]
    xt = x.T.contiguous()
    check_values(q.qmm_fp4_quantize(x, block=block), x)
    check_values(q.qmm_fp4_quantize(x, block=block, transpose=True), xt)
    a, b = q.qmm_fp4_quantize_both(x, block=block)
    check_values(a, x)
    check_values(b, xt)


@pytest.mark.parametrize("R,C,ld", [(1217, 8208, 8208), (1300, 11008, 11016), (1400, 13200, 13200)])
def test_quantise_many_long_rows(R, C, ld):
    """Rows that go through shared memory: the values, a row of zeros, non-finite ones, and the bytes of the
    same rows packed a few at a time."""
    x = make(R, ld, torch.bfloat16, C)
    x[7] = 0
    x[64, 5], x[R - 1, C - 1] = float("nan"), float("inf")
    x = x[:, :C]
    m = q.qmm_fp4_quantize(x, block=16)
    q.check_device_error()
    y = q.qmm_fp4_dequantize(m, out_dtype=torch.float32)
    for r in (0, 128, 1152):
        part = q.qmm_fp4_dequantize(q.qmm_fp4_quantize(x[r:r + 60], block=16), out_dtype=torch.float32)
        assert torch.equal(torch.nan_to_num(y[r:r + 60], nan=-7.0), torch.nan_to_num(part, nan=-7.0))
    assert (y[7] == 0).all() and torch.isnan(y[64]).all() and torch.isnan(y[R - 1]).all()
    rows = [0, 1, 31, 32, 63, 65, 127, 128, 777, R - 2]
    want = O.fp4_values(f32(x[rows]), 16, False)
    assert np.array_equal(y[rows].cpu().numpy(), want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32])
def test_zeros_extremes_and_non_finite(dt, block):
    t = TYPES[dt]
    x = make(140, 320, t, 9)
    x[0] = 0
    x[1] = torch.finfo(t).tiny
    x[2] = torch.finfo(t).tiny / 32
    x[3] = torch.finfo(t).max
    x[4, ::2] = -torch.finfo(t).max
    x[5, :32] = 0
    x[6] = 1e-30
    x[7, 100] = float("inf")
    x[8, 319] = float("nan")
    x[139, 5] = float("-inf")
    x[10] = -0.0
    for v in (x, x.T.contiguous()):
        check_values(q.qmm_fp4_quantize(v, block=block), v)
        a, b = q.qmm_fp4_quantize_both(v, block=block)
        check_values(a, v)
        check_values(b, v.T.contiguous())
        check_values(q.qmm_fp4_quantize(v, block=block, transpose=True), v.T.contiguous())


@pytest.mark.parametrize("block", [16, 32])
def test_every_tie_and_code(block):
    """Multiples of an eighth under a fixed block maximum: every code and every midpoint, both signs."""
    k = torch.arange(-48, 49, device="cuda").float() / 8
    x = torch.zeros(4, 13 * 32, device="cuda")
    for i in range(97):
        x[0, (i // 8) * 32 + 1 + i % 8] = k[i]
    x[0, ::16] = 6.0
    x[1] = x[0] * 2.0 ** -20
    x[2] = x[0] * 2688.0 / 6
    x[3] = x[0] * 3.0
    for t in (torch.float32, torch.bfloat16):
        check_values(q.qmm_fp4_quantize(x.to(t), block=block), x.to(t))
        check_values(q.qmm_fp4_quantize(x.to(t).T.contiguous(), block=block, transpose=True), x.to(t))


def check_product(a, b, block, out, got, rows=None):
    A, B = f32(a), f32(b)
    if rows is not None:
        A, got = A[rows], got[rows]
    exact, mag = O.fp4_matmul(A, B, block)
    K = A.shape[1]
    # K / 64 accumulations, each (and the sum of 64 products in it) exact to 2^-22 of the magnitudes
    # summed, then two scale factors
    bound = (K / 64 + 16) * 2.0 ** -22 * mag
    g = f32(got).astype(np.float64)
    mant = 7 if out == torch.bfloat16 else 23
    err = np.abs(g - exact)
    lim = bound + half_ulp(exact, mant) * 1.01
    assert (err <= lim).all(), f"{(err > lim).sum()} of {err.size} out of bound, worst {(err / lim).max():.3g}"


PRODUCTS = [(1, 1, 1), (1, 64, 128), (3, 33, 100), (8, 128, 64), (16, 1000, 4100), (17, 129, 513), (64, 300, 2048),
            (100, 640, 1024), (128, 128, 256), (129, 257, 640), (200, 1111, 300), (256, 256, 512), (257, 500, 1000),
            (300, 1024, 4096), (513, 777, 384), (1, 4096, 8192), (40, 2048, 16384)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_matmul(M, N, K, out, block):
    a, b = make(M, K, torch.bfloat16, M + K), make(N, K, torch.float32, N + K)
    A, B = q.qmm_fp4_quantize(a, block=block), q.qmm_fp4_quantize(b, block=block)
    y = q.qmm_fp4_matmul(A, B, out_dtype=out)
    q.check_device_error()
    assert q.last_kernel().startswith("gemm_fp4")
    check_product(a, b, block, out, y)
    assert torch.equal(y, q.qmm_fp4_matmul(A, B, out_dtype=out))


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,N,K", [(2000, 1536, 1024), (700, 5000, 2176), (1, 28672, 8192), (150, 11007, 4100)])
def test_matmul_many_tiles(M, N, K, block):
    a, b = make(M, K, torch.bfloat16, 1), make(N, K, torch.bfloat16, 2)
    y = q.qmm_fp4_matmul(q.qmm_fp4_quantize(a, block=block), q.qmm_fp4_quantize(b, block=block))
    q.check_device_error()
    rows = np.unique(np.concatenate([np.arange(0, M, max(1, M // 40)), [M - 1]]))
    check_product(a, b, block, torch.bfloat16, y, rows)


@pytest.mark.parametrize("block", [16, 32])
def test_a_row_uses_its_own_operands_only(block):
    """NaN rows of either operand stay in their rows and columns of the product; a padded tile's
    unwritten rows reach nothing."""
    a, b = make(130, 200, torch.bfloat16, 3), make(70, 200, torch.bfloat16, 4)
    clean = q.qmm_fp4_matmul(q.qmm_fp4_quantize(a, block=block), q.qmm_fp4_quantize(b, block=block))
    a[5, 17], b[69, 199] = float("nan"), float("inf")
    for fill in (0, 255, 127):
        mats = []
        for t in (a, b):
            m = q.Fp4Matrix(torch.full((q.qmm_fp4_bytes(*t.shape, block),), fill, dtype=torch.uint8, device="cuda"),
                            *t.shape, block)
            mats.append(q.qmm_fp4_quantize(t, block=block, out=m))
        y = q.qmm_fp4_matmul(*mats)
        nan = torch.zeros_like(y, dtype=torch.bool)
        nan[5], nan[:, 69] = True, True
        assert torch.equal(torch.isnan(y), nan)
        assert torch.equal(y[~nan], clean[~nan])


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,K,N", [(65, 130, 200), (300, 257, 129), (512, 640, 384)])
def test_training_step(M, K, N, block):
    """y, dx and dw of a linear layer, each operand packed along the axis its product sums over."""
    x, w, dy = make(M, K, torch.bfloat16, 5), make(N, K, torch.bfloat16, 6), make(M, N, torch.bfloat16, 7)
    xq, xt = q.qmm_fp4_quantize_both(x, block=block)
    wq, wt = q.qmm_fp4_quantize_both(w, block=block)
    dq, dt = q.qmm_fp4_quantize_both(dy, block=block)
    check_product(x, w, block, torch.float32, q.qmm_fp4_matmul(xq, wq, out_dtype=torch.float32))
    check_product(dy, w.T.contiguous(), block, torch.float32, q.qmm_fp4_matmul(dq, wt, out_dtype=torch.float32))
    check_product(dy.T.contiguous(), x.T.contiguous(), block, torch.float32,
                  q.qmm_fp4_matmul(dt, xt, out_dtype=torch.float32))
    q.check_device_error()


def test_gradients_against_differences():
    """With operands that 4 bits hold exactly, dx and dw are the differences of the layer's own outputs."""
    M, K, N = 40, 96, 64
    rng = np.random.default_rng(0)
    codes = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -.5, -1, -2, -3, -6], np.float32)
    x, w, dy = (rng.choice(codes, s).astype(np.float32) for s in ((M, K), (N, K), (M, N)))
    for t in (x, w, dy):
        t[:, ::16] = 6.0
        t[::16, :] = 6.0
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731

    def layer(xv, wv):
        return q.qmm_fp4_matmul(q.qmm_fp4_quantize(dev(xv), block=32), q.qmm_fp4_quantize(dev(wv), block=32),
                                out_dtype=torch.float32).cpu().numpy().astype(np.float64)
    (_, xt), (_, wt), (dq, dt) = (q.qmm_fp4_quantize_both(dev(t), block=32) for t in (x, w, dy))
    dx = q.qmm_fp4_matmul(dq, wt, out_dtype=torch.float32).cpu().numpy()
    dw = q.qmm_fp4_matmul(dt, xt, out_dtype=torch.float32).cpu().numpy()
    base = (layer(x, w) * dy).sum()
    for i, k in ((3, 7), (0, 1), (39, 95), (20, 50)):       # one element a code further: exact in 4 bits
        for j, (t, grad) in enumerate(((x, dx), (w, dw))):
            v = t.copy()
            step = 2.0 if v[i, k] == 4.0 else -4.0 if v[i, k] == 6.0 else 6.0 - v[i, k]
            if v[i, k] == 6.0:
                step = -2.0
            v[i, k] += step
            diff = (layer(*((v, w) if j == 0 else (x, v))) * dy).sum() - base
            assert diff == pytest.approx(grad[i, k] * step, rel=1e-5, abs=1e-3)


def test_empty_operands():
    z = torch.zeros(0, 64, device="cuda")
    a = q.qmm_fp4_quantize(z)
    b = q.qmm_fp4_quantize(torch.ones(5, 64, device="cuda"))
    assert q.qmm_fp4_matmul(a, b).shape == (0, 5) and q.qmm_fp4_matmul(b, a).shape == (5, 0)
    assert q.qmm_fp4_dequantize(a).shape == (0, 64)
    k0 = q.qmm_fp4_quantize(torch.ones(5, 0, device="cuda"))
    assert (q.qmm_fp4_matmul(k0, k0, out_dtype=torch.float32) == torch.zeros(5, 5, device="cuda")).all()


def test_other_stream_graph_and_reused_buffers():
    x, w = make(70, 512, torch.bfloat16, 1), make(384, 512, torch.bfloat16, 2)
    W = q.qmm_fp4_quantize(w)
    want = q.qmm_fp4_matmul(q.qmm_fp4_quantize(x), W)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = q.qmm_fp4_matmul(q.qmm_fp4_quantize(x), W)
    s.synchronize()
    assert torch.equal(got, want)
    xs = torch.zeros_like(x)
    buf, bt = q.qmm_fp4_quantize_both(xs)
    y = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qmm_fp4_quantize_both(xs, out=buf, out_t=bt)
        q.qmm_fp4_matmul(buf, W, out=y)
    for src in (x, torch.flip(x, (0,))):
        xs.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, q.qmm_fp4_matmul(q.qmm_fp4_quantize(src), W))


def test_offsets_past_32_bits():
    R, C = 140000, 16384
    x = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [0, 70000, 131073, R - 1]
    for r in rows:
        x[r] = torch.randn(C, generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.tensor(rows, device="cuda")
    want = O.fp4_values(f32(x[idx]), 16, True)
    m = q.qmm_fp4_quantize(x)
    y = q.qmm_fp4_dequantize(m)
    assert np.array_equal(f32(y[idx]), want) and not y[1:70000].any()
    del y
    w = torch.randn(100, C, generator=g, device="cuda")
    p = q.qmm_fp4_matmul(m, q.qmm_fp4_quantize(w))
    q.check_device_error()
    check_product(x[idx], w, 16, torch.bfloat16, p[idx])
    del m, p
    t = q.qmm_fp4_quantize(x, block=32, transpose=True)
    back = q.qmm_fp4_dequantize(t)
    cols = [0, 9999, C - 1]
    sub = x[:, cols].T.contiguous()
    assert np.array_equal(f32(back[cols]), O.fp4_values(f32(sub), 32, True))
    del back, t, x
    torch.cuda.empty_cache()
