"""qmm_rms_norm_s8 on finite rows whose squares leave float32's range (from above, or
from below where eps does not cover them): the scale and rstd of the definition, in
every form of the kernel, with ordinary rows beside them; and the gradient of such rows."""
import numpy as np
import pytest
import torch

from test_gpu_rms_norm import check_backward, check_forward, f32

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# the magnitude of a row's elements (1: ordinary)
LARGE = [3e19, 1.0, 2e19, 1e25, 1e30, 5e36, 2.0, 1e18]
SMALL = [1e-24, 1.0, 2.0 ** -70, 2.0 ** -63, 1e-28, 2.0 ** -75, 1e-18, 2.0 ** -90]


def rows(magnitudes, H, dt, seed, M=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.tensor(magnitudes, dtype=torch.float64, device="cuda")
    m = m.repeat((M or len(magnitudes)) // len(magnitudes) + 1)[:M or len(magnitudes)]
    x = (torch.randn(m.numel(), H, generator=g, device="cuda").double() * m[:, None]).to(dt)
    return x, (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dt)


# widths of one vector a thread, several, odd ones, one warp a row, rows read twice
WIDTHS = [7, 64, 1000, 4096, 5003, 40000, 131072]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("magnitudes,eps", [(LARGE, 1e-6), (LARGE, 0.0), (SMALL, 0.0), (SMALL, 2.0 ** -133),
                                            (SMALL, 2.0 ** -119), (SMALL, 2.0 ** -121)])
def test_squares_out_of_range(H, dt, magnitudes, eps):
    x, w = rows(magnitudes, H, TYPES[dt], H)
    out = q.qmm_rms_norm_s8(x, w, eps=eps, save_rstd=True)
    assert (out.scale > 0).all() and torch.isfinite(out.scale).all()
    check_forward(x, None, w, out, eps)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", WIDTHS)
def test_with_a_residual_in_place(H, dt):
    x, w = rows(LARGE + SMALL, H, TYPES[dt], H + 1)
    r = (x.double() * 0.25).to(x.dtype).flip(1)
    for dst in (None, 0, 1):
        a, b = x.clone(), r.clone()
        out = q.qmm_rms_norm_s8(a, w, residual=b, eps=0.0, h_out=None if dst is None else (a, b)[dst], save_rstd=True)
        check_forward(x, r, w, out, 0.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,H", [(700, 256), (700, 4096), (700, 5003), (330, 20000)])
def test_many_rows(M, H, dt):
    for magnitudes in (LARGE, SMALL):
        x, w = rows(magnitudes, H, TYPES[dt], H + 2, M)
        check_forward(x, None, w, q.qmm_rms_norm_s8(x, w, eps=0.0, save_rstd=True), 0.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_that_are_still_marked(dt):
    """Zeros, an infinity and a NaN beside squares that overflow; a product with the weight that overflows."""
    x, w = rows([3e19] * 6, 1024, TYPES[dt], 4)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 9] = float("nan")
    x[3, 100] = 3e38
    w[100] = 4.0
    out = q.qmm_rms_norm_s8(x, w, eps=0.0, save_rstd=True)
    assert out.scale[0].item() == 1.0 and torch.isnan(out.scale[1:4]).all() and (out.q[:4] == 0).all()
    check_forward(x[4:], None, w, q.RmsNormS8(out.q[4:], out.scale[4:], x[4:], out.rstd[4:]), 0.0)
    assert out.rstd[3].item() == pytest.approx(1 / np.sqrt((f32(x[3]).astype(np.float64) ** 2).mean()), rel=1e-5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,H", [(9, 4096), (33, 5003), (12, 64)])
def test_gradient_of_large_rows(M, H, dt):
    t = TYPES[dt]
    h, w = rows(LARGE, H, t, 5, M)
    g = torch.Generator(device="cuda").manual_seed(6)
    dy = torch.randn(M, H, generator=g, device="cuda").to(t)
    rstd = q.qmm_rms_norm_s8(h, w, save_rstd=True).rstd
    dx, dw = q.qmm_rms_norm_backward(dy, h, w, rstd)
    check_backward(dy, h, w, rstd, None, dx, dw)
    assert (dx != 0).any(dim=1).all()
