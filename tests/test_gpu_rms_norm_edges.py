"""The norm's gradient of rows off 16 bytes whose tensors end where other memory begins:
what lies behind the last row (NaN here) reaches nothing, whether that row is the first of
its CTA's, one that its ring holds from the start, or one that is copied in later."""
import pytest
import torch

from test_gpu_rms_norm import check_backward

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def ends_before_nan(M, H, dt, g):
    """[M, H] contiguous, followed by NaN in the same allocation."""
    flat = torch.full((M * H + 64,), float("nan"), dtype=dt, device="cuda")
    t = flat[:M * H].view(M, H)
    t.copy_(torch.randn(M, H, generator=g, device="cuda"))
    return t


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("with_dh", [True, False])
@pytest.mark.parametrize("M,H", [(1, 1001), (5, 1003), (151, 4099), (153, 5003), (309, 2053), (1601, 4101), (1700, 4095),
                                 (1217, 8189), (2435, 1019), (1500, 12283), (333, 16381)])
def test_last_row(M, H, dt, with_dh):
    g = torch.Generator(device="cuda").manual_seed(M + H)
    t = TYPES[dt]
    h, dy = ends_before_nan(M, H, t, g), ends_before_nan(M, H, t, g)
    dh = ends_before_nan(M, H, t, g) if with_dh else None
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(t)
    rstd = torch.rsqrt((h.float() ** 2).mean(dim=1))
    dx, dw = q.qmm_rms_norm_backward(dy, h, w, rstd, dh=dh)
    q.check_device_error()
    rows = slice(max(0, M - 400), M)
    assert torch.isfinite(dx.float()).all() and torch.isfinite(dw).all()
    # (the gradient's rows are their own; dweight from all of them)
    sub, _ = q.qmm_rms_norm_backward(dy[rows], h[rows], w, rstd[rows].contiguous(), dh=None if dh is None else dh[rows])
    check_backward(dy, h, w, rstd, dh, dx, dw)
    err = (sub.double() - dx[rows].double()).abs()
    assert (err <= (2.0 ** -7 if dt == "bf16" else 2.0 ** -20) * (1 + dx[rows].double().abs())).all()
