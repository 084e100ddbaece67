"""Rows without elements: the scale of a row of zeros, and no memory left as it was found."""
import pytest
import torch

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")


@pytest.mark.parametrize("given", [False, True])
def test_rows_without_elements(given):
    s = torch.cuda.Stream() if given else None
    for _ in range(4):
        with torch.cuda.stream(s):
            junk = [torch.full((n,), 7.0, device="cuda") for n in (5, 5, 64, 64)]   # what the call's blocks held
        torch.cuda.synchronize()
        del junk
        x = torch.empty(5, 0, device="cuda", dtype=torch.bfloat16)
        n = q.qmm_rms_norm_s8(x, torch.empty(0, device="cuda"), residual=x, save_rstd=True, stream=s)
        torch.cuda.synchronize()
        assert n.q.shape == (5, 0) and n.h.shape == (5, 0)
        assert (n.scale == 1).all() and torch.isnan(n.rstd).all()      # (the mean of no squares)
        assert q.qmm_s8_dequantize_rows(n.q, n.scale).shape == (5, 0)
        dx, dw = q.qmm_rms_norm_backward(x, n.h, torch.empty(0, device="cuda"), n.rstd, stream=s)
        assert dx.shape == (5, 0) and dw.shape == (0,)
