"""qmm_rms_norm_s8, qmm_s8_dequantize_rows and qmm_rms_norm_backward against the
oracle: the int8 rows and h bit for bit, scales, statistics and gradients within
bounds derived from fp32 summation. Widths around every vector and CTA boundary,
strided and unaligned rows, in-place sums, empty and non-finite rows, offsets
past 32 bits, other streams, CUDA graphs, and the feeding of qmm_a8w8."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as O
from _helpers import half_ulp

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")

U = 2.0 ** -24   # half an ulp of 1 in float32
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def f32(t):
    return t.float().cpu().numpy()


def make(M, H, dt, seed, residual=True, w_dt=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, H, generator=g, device="cuda")
    x = (x * torch.where(torch.rand(M, H, generator=g, device="cuda") < 0.01, 20.0, 1.0)).to(dt)
    r = (3 * torch.randn(M, H, generator=g, device="cuda")).to(dt) if residual else None
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(w_dt or dt)
    return x, r, w


def check_forward(x, r, w, out, eps):
    bf = x.dtype == torch.bfloat16
    wq, ws, wh, wr = O.rms_norm_s8(f32(x), f32(w), None if r is None else f32(r), eps, bf)
    H = x.shape[1]
    assert np.array_equal(f32(out.h), wh, equal_nan=True)
    got = out.q.cpu().numpy()
    assert np.array_equal(got, wq), f"{(got != wq).sum()} of {wq.size} int8 values differ"
    # a sum of H squares (relative error below 40 + H / 64 half-ulps for any order with 64 or more
    # parallel sums of at most H / 64), the root, and four roundings
    tol = U * (48 + H / 64)
    s = out.scale.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(s), np.isnan(ws))
    ok = ~np.isnan(ws)
    assert (np.abs(s - ws)[ok] <= tol * np.abs(ws[ok])).all()
    if out.rstd is not None:
        rs = out.rstd.cpu().numpy().astype(np.float64)
        assert (np.abs(rs - wr)[ok] <= tol * wr[ok]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("M,H", [(1, 1), (3, 7), (5, 8), (2, 33), (9, 64), (4, 100), (17, 255), (8, 256), (3, 1000),
                                 (1, 4096), (33, 4096), (7, 5003), (5, 8192), (2, 11008), (3, 16384), (2, 40000),
                                 (1, 131072), (2, 70001), (700, 251), (701, 4099), (900, 13), (400, 8190), (40, 4097)])
def test_forward(M, H, dt, residual):
    x, r, w = make(M, H, TYPES[dt], M * 1000 + H, residual)
    out = q.qmm_rms_norm_s8(x, w, residual=r, eps=1e-5, save_rstd=True)
    assert q.last_kernel().startswith("rms_norm_s8")
    check_forward(x, r, w, out, 1e-5)
    for o in (torch.float32, torch.bfloat16):   # read back: one product, one rounding
        y = q.qmm_s8_dequantize_rows(out.q, out.scale, out_dtype=o)
        want = (out.q.float() * out.scale[:, None]).to(o)
        assert torch.equal(y, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("other", ["bf16", "f32"])
def test_forward_many_rows_and_weight_types(dt, other):
    x, r, w = make(3001, 768, TYPES[dt], 5, True, TYPES[other])
    check_forward(x, r, w, q.qmm_rms_norm_s8(x, w, residual=r), 1e-6)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("ld,off", [(4096 + 8, 0), (4096 + 3, 0), (4096 + 16, 1), (8192, 5)])
def test_forward_strides_and_alignment(dt, ld, off):
    M, H = 6, 4096
    x, r, w = make(M, ld + off, TYPES[dt], 11)
    xs, rs = x[:, off:off + H], r[:, off:off + H]
    out = q.qmm_rms_norm_s8(xs, w[:H].contiguous(), residual=rs)
    check_forward(xs, rs, w[:H], out, 1e-6)
    # one operand aligned, the other not
    out = q.qmm_rms_norm_s8(xs.contiguous(), w[:H].contiguous(), residual=rs)
    check_forward(xs, rs, w[:H], out, 1e-6)


@pytest.mark.parametrize("H", [4096, 5003, 70000])
def test_sum_in_place(H):
    """h over x, or over the residual."""
    x, r, w = make(5, H, torch.bfloat16, 2)
    want = q.qmm_rms_norm_s8(x, w, residual=r)
    for which in (0, 1):
        a, b = x.clone(), r.clone()
        dst = (a, b)[which]
        got = q.qmm_rms_norm_s8(a, w, residual=b, h_out=dst)
        assert got.h is dst
        assert torch.equal(dst, want.h) and torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_empty_zero_and_non_finite_rows(dt):
    t = TYPES[dt]
    x, r, w = make(8, 1024, t, 3)
    x[0], r[0] = 0, 0
    x[1, 5] = float("inf")
    x[2, 1023] = float("nan")
    x[3, 7], r[3, 7] = float("inf"), float("-inf")
    x[4] = torch.finfo(t).tiny
    r[4] = 0
    x[5], r[5] = torch.finfo(t).tiny / 64, 0          # subnormal
    x[6], r[6] = 1e15, 0
    w[9] = 0
    out = q.qmm_rms_norm_s8(x, w, residual=r)
    check_forward(x, r, w, out, 1e-6)
    assert out.scale[0].item() == 1.0 and torch.isnan(out.scale[1:4]).all() and not torch.isnan(out.scale[4:]).any()
    assert (out.q[1:4] == 0).all()
    w0 = torch.zeros_like(w)
    z = q.qmm_rms_norm_s8(x[7:8], w0, residual=r[7:8])
    assert (z.q == 0).all() and z.scale.item() == 1.0
    e = q.qmm_rms_norm_s8(x[:0], w, residual=r[:0])
    assert e.q.shape == (0, 1024) and q.qmm_s8_dequantize_rows(e.q, e.scale).shape == (0, 1024)


def test_offsets_past_32_bits():
    M, H = 140000, 16384          # 2.29e9 elements
    x = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    x.view(-1)[:].fill_(0.5)
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [0, 70000, 131073, M - 1]
    for m in rows:
        x[m] = torch.randn(H, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    out = q.qmm_rms_norm_s8(x, w, save_rstd=True)
    idx = torch.tensor(rows, device="cuda")
    sub = q.RmsNormS8(out.q[idx], out.scale[idx], x[idx], out.rstd[idx])
    check_forward(x[idx], None, w, sub, 1e-6)
    y = q.qmm_s8_dequantize_rows(out.q, out.scale)
    assert torch.equal(y[idx], (out.q[idx].float() * out.scale[idx][:, None]).bfloat16())
    del y, out
    dy = torch.full((M, H), 0.25, dtype=torch.bfloat16, device="cuda")
    rstd = torch.rsqrt(torch.full((M,), 0.25, device="cuda"))
    dx, _ = q.qmm_rms_norm_backward(dy, x, w, rstd)
    want, _ = O.rms_norm_backward(f32(dy[idx]), f32(x[idx]), f32(w), rstd[idx].cpu().numpy())
    err = np.abs(dx[idx].float().cpu().numpy() - want)
    assert (err <= 1e-4 + half_ulp(want, 7)).all()
    torch.cuda.empty_cache()


def check_backward(dy, h, w, rstd, dh, dx, dw):
    M, H = h.shape
    want, wantw = O.rms_norm_backward(f32(dy), f32(h), f32(w), rstd.cpu().numpy(), None if dh is None else f32(dh))
    r = rstd.cpu().numpy().astype(np.float64)[:, None]
    n = np.abs(f32(h).astype(np.float64)) * r
    g = np.abs(f32(dy).astype(np.float64) * f32(w).astype(np.float64))
    # the mean: a sum of H terms in at least 32 parallel sums; then a handful of roundings
    bound = r * (8 * U * g + n * ((48 + H / 32) * U * (g * n).mean(axis=1, keepdims=True)))
    if dh is not None:
        bound = bound + 2 * U * (np.abs(f32(dh)) + np.abs(want))
    got = dx.float().cpu().numpy().astype(np.float64)
    mant = 7 if dx.dtype == torch.bfloat16 else 23
    err = np.abs(got - want)
    assert (err <= bound + 1.01 * half_ulp(want, mant) + 1e-38).all(), float((err / (bound + half_ulp(want, mant))).max())
    boundw = (8 + M) * U * np.abs(f32(dy).astype(np.float64) * n).sum(axis=0)
    errw = np.abs(dw.cpu().numpy().astype(np.float64) - wantw)
    assert (errw <= boundw + 1e-38).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("with_dh", [True, False])
@pytest.mark.parametrize("M,H", [(1, 1), (3, 5), (1, 4096), (40, 33), (300, 256), (5, 1000), (1000, 4096), (33, 5003),
                                 (777, 64), (20, 11008), (9, 16384), (3, 40000), (2, 100001), (2000, 251), (3000, 13), (1500, 4099), (700, 8190),
                                 (310, 1025), (161, 12285)])
def test_backward(M, H, dt, with_dh):
    t = TYPES[dt]
    g = torch.Generator(device="cuda").manual_seed(M + H)
    h, _, w = make(M, H, t, M + 7 * H, False)
    dy = torch.randn(M, H, generator=g, device="cuda").to(t)
    dh = torch.randn(M, H, generator=g, device="cuda").to(t) if with_dh else None
    rstd = q.qmm_rms_norm_s8(h, w, save_rstd=True).rstd
    dx, dw = q.qmm_rms_norm_backward(dy, h, w, rstd, dh=dh)
    assert q.last_kernel().startswith("rms_norm_backward")
    check_backward(dy, h, w, rstd, dh, dx, dw)
    dx2, dw2 = q.qmm_rms_norm_backward(dy, h, w, rstd, dh=dh)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)     # the order of the sums is fixed


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward_strides_weight_types_and_in_place(dt):
    t = TYPES[dt]
    M, H = 37, 1024
    g = torch.Generator(device="cuda").manual_seed(4)
    big = torch.randn(M, 3 * H + 5, generator=g, device="cuda").to(t)
    h, dy, dh = big[:, 3:H + 3], big[:, H + 4:2 * H + 4], big[:, 2 * H + 5:]
    for wt in (torch.float32, torch.bfloat16):
        w = torch.randn(H, generator=g, device="cuda").to(wt)
        rstd = torch.rsqrt((h.float() ** 2).mean(dim=1))
        dx, dw = q.qmm_rms_norm_backward(dy, h, w, rstd, dh=dh)
        check_backward(dy, h, w, rstd, dh, dx, dw)
        for which in (0, 1):
            a, b = dy.contiguous(), dh.contiguous()
            got, gw = q.qmm_rms_norm_backward(a, h, w, rstd, dh=b, out=(a, b)[which])
            assert torch.equal(got, dx) and torch.equal(gw, dw)


def test_backward_of_no_rows_is_zero():
    w = torch.ones(300, device="cuda")
    e = torch.empty(0, 300, device="cuda")
    dx, dw = q.qmm_rms_norm_backward(e, e, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 300) and (dw == 0).all()


def test_gradient_against_differences():
    """The forward's own outputs: q * scale moves as the gradient says, within the quantiser's steps."""
    M, H = 4, 512
    rng = np.random.default_rng(0)
    h, w = rng.standard_normal((M, H)).astype(np.float32), (1 + 0.1 * rng.standard_normal(H)).astype(np.float32)
    dy = rng.standard_normal((M, H)).astype(np.float32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    rstd = q.qmm_rms_norm_s8(dev(h), dev(w), eps=1e-6, save_rstd=True).rstd
    dx, dw = q.qmm_rms_norm_backward(dev(dy), dev(h), dev(w), rstd)
    loss = lambda hh, ww: (O.rms_norm(hh, ww, 1e-6) * dy).sum()  # noqa: E731
    t = 1e-5
    for seed in range(8):
        d = np.random.default_rng(seed).standard_normal((M, H))
        num = (loss(h + t * d, w) - loss(h - t * d, w)) / (2 * t)
        assert abs(num - (dx.cpu().numpy() * d).sum()) < 1e-4 * np.sqrt(M * H)
        d = np.random.default_rng(seed).standard_normal(H)
        num = (loss(h, w + t * d) - loss(h, w - t * d)) / (2 * t)
        assert abs(num - (dw.cpu().numpy() * d).sum()) < 1e-4 * np.sqrt(M * H)


def test_other_stream_and_graph():
    x, r, w = make(64, 2048, torch.bfloat16, 8)
    want = q.qmm_rms_norm_s8(x, w, residual=r)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = q.qmm_rms_norm_s8(x, w, residual=r, save_rstd=True)
        y = q.qmm_s8_dequantize_rows(got.q, got.scale)
        dx, dw = q.qmm_rms_norm_backward(y, got.h, w, got.rstd, dh=r)
    s.synchronize()
    assert torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale) and torch.equal(got.h, want.h)
    x2, r2 = torch.zeros_like(x), torch.zeros_like(r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = q.qmm_rms_norm_s8(x2, w, residual=r2, save_rstd=True)
        y2 = q.qmm_s8_dequantize_rows(out.q, out.scale)
        dx2, dw2 = q.qmm_rms_norm_backward(y2, out.h, w, out.rstd, dh=r2)
    x2.copy_(x)
    r2.copy_(r)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.q, want.q) and torch.equal(y2, y) and torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_feeds_a8w8():
    """norm -> qmm_a8w8: the product of the normalised rows within the quantisers' steps."""
    M, H, N = 300, 512, 256
    x, r, w = make(M, H, torch.bfloat16, 21)
    g = torch.Generator(device="cuda").manual_seed(0)
    W = torch.randint(-127, 128, (H, N), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=g, device="cuda") * 1e-3
    n = q.qmm_rms_norm_s8(x, w, residual=r)
    y = q.qmm_a8w8(n.q, W, n.scale, ws, out_dtype=torch.float32)
    q.check_device_error()
    exact = O.rms_norm(f32(n.h), f32(w), 1e-6) @ (W.cpu().numpy().astype(np.float64) * ws.cpu().numpy())
    step = n.scale.cpu().numpy().astype(np.float64)[:, None] * 0.5001
    bound = step * np.abs(W.cpu().numpy().astype(np.float64) * ws.cpu().numpy()).sum(axis=0)
    assert (np.abs(y.cpu().numpy() - exact) <= bound).all()
