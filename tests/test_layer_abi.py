"""Refusals of the norm's and the 4-bit entry points, on the host, without a GPU."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(260)


@pytest.fixture(scope="module")
def qmm():
    import quantized_int8_matmul_gb300 as q
    lib = q.lib()
    i64, vp, ci, sz, cf = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    lib.qmm_rms_norm_s8.argtypes = [vp, ci, i64, i64, i64, vp, i64, vp, ci, cf, vp, vp, vp, vp, vp]
    lib.qmm_s8_dequantize_rows.argtypes = [vp, vp, i64, i64, vp, ci, vp]
    lib.qmm_rms_norm_backward.argtypes = [vp, i64, vp, i64, vp, i64, ci, i64, i64, vp, ci, vp, vp, vp, vp, sz, vp]
    lib.qmm_fp4_quantize.argtypes = [vp, ci, i64, i64, i64, ci, ci, vp, sz, vp]
    lib.qmm_fp4_quantize_both.argtypes = [vp, ci, i64, i64, i64, ci, vp, sz, vp, sz, vp]
    lib.qmm_fp4_dequantize.argtypes = [vp, sz, i64, i64, ci, vp, ci, vp]
    lib.qmm_fp4_matmul.argtypes = [vp, sz, i64, vp, sz, i64, i64, ci, vp, ci, vp]
    return q


def test_rms_norm_refusals(qmm):
    lib, bad = qmm.lib(), qmm.QMM_ERR_INVALID_ARG

    def call(x=P, xd=qmm.QMM_BF16, M=4, H=64, ldx=64, r=P, ldr=64, w=P, wd=qmm.QMM_BF16, eps=1e-6, h=None, q=P, s=P,
             rs=P):
        return lib.qmm_rms_norm_s8(x, xd, M, H, ldx, r, ldr, w, wd, eps, h, q, s, rs, None)
    for kw in (dict(xd=qmm.QMM_S8), dict(wd=qmm.QMM_S32), dict(M=-1), dict(H=2 ** 31), dict(ldx=63), dict(ldr=63),
               dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(w=None), dict(q=None), dict(s=None),
               dict(h=P, x=P, ldx=65)):
        assert call(**kw) == bad, kw
    assert call(M=0, x=None) == qmm.QMM_OK and call(H=0, ldx=0, ldr=0) == qmm.QMM_OK
    assert lib.qmm_s8_dequantize_rows(P, P, 4, 4, P, qmm.QMM_S8, None) == bad
    assert lib.qmm_s8_dequantize_rows(None, P, 4, 4, P, qmm.QMM_F32, None) == bad
    assert lib.qmm_s8_dequantize_rows(None, None, 0, 4, None, qmm.QMM_F32, None) == qmm.QMM_OK


def test_rms_norm_backward_refusals(qmm):
    lib, bad = qmm.lib(), qmm.QMM_ERR_INVALID_ARG
    need = lib.qmm_rms_norm_backward_workspace_bytes(4, 64)
    assert need >= 64 * 4 and lib.qmm_rms_norm_backward_workspace_bytes(-1, 64) == 0

    def call(dy=P, lddy=64, h=P, ldh=64, dh=None, lddh=64, dt=qmm.QMM_F32, M=4, H=64, w=P, wd=qmm.QMM_F32, r=P,
             dx=ctypes.c_void_p(512), dw=P, ws=P, wb=need):
        return lib.qmm_rms_norm_backward(dy, lddy, h, ldh, dh, lddh, dt, M, H, w, wd, r, dx, dw, ws, wb, None)
    for kw in (dict(dt=qmm.QMM_U8), dict(wd=qmm.QMM_U8), dict(M=-1), dict(lddy=1), dict(ldh=1), dict(dh=P, lddh=1),
               dict(dy=None), dict(h=None), dict(w=None), dict(r=None), dict(dx=None), dict(dw=None), dict(ws=None),
               dict(ws=ODD), dict(wb=need - 1), dict(dx=P, lddy=65), dict(dx=P, dy=ctypes.c_void_p(1024))):
        assert call(**kw) == bad, kw
    assert call(H=0, lddy=0, ldh=0) == qmm.QMM_OK


def test_fp4_refusals(qmm):
    lib, bad, F = qmm.lib(), qmm.QMM_ERR_INVALID_ARG, qmm.QMM_F32
    need = lib.qmm_fp4_bytes(100, 200, 16)
    assert need == 1 * 2 * (8192 + 1024) + 1024 and lib.qmm_fp4_bytes(100, 200, 32) == 2 * (8192 + 512)
    assert lib.qmm_fp4_bytes(100, 200, 8) == 0 and lib.qmm_fp4_bytes(-1, 200, 16) == 0
    assert lib.qmm_fp4_bytes(2 ** 31 - 1, 2 ** 31 - 1, 16) == 0 and lib.qmm_fp4_bytes(0, 5, 16) == 0

    def quant(x=P, xd=F, r=100, c=200, ld=200, tr=0, bl=16, p=P, pb=need):
        return lib.qmm_fp4_quantize(x, xd, r, c, ld, tr, bl, p, pb, None)
    for kw in (dict(xd=qmm.QMM_S8), dict(r=-1), dict(ld=199), dict(tr=2), dict(bl=64), dict(x=None), dict(p=None),
               dict(p=ODD), dict(pb=need - 1), dict(tr=1, ld=99)):
        assert quant(**kw) == bad, kw
    assert quant(r=2 ** 31 - 1, c=2 ** 31 - 1, ld=2 ** 31) == qmm.QMM_ERR_UNSUPPORTED
    assert quant(r=0, p=None) == qmm.QMM_OK

    def both(p=P, pb=need, t=P, tb=lib.qmm_fp4_bytes(200, 100, 16), bl=16):
        return lib.qmm_fp4_quantize_both(P, F, 100, 200, 200, bl, p, pb, t, tb, None)
    for kw in (dict(p=None), dict(t=None), dict(t=ODD), dict(pb=0), dict(tb=100), dict(bl=0)):
        assert both(**kw) == bad, kw

    def deq(p=P, pb=need, r=100, c=200, bl=16, y=P, yd=F):
        return lib.qmm_fp4_dequantize(p, pb, r, c, bl, y, yd, None)
    for kw in (dict(p=None), dict(pb=need - 1), dict(r=129), dict(bl=4), dict(y=None), dict(yd=qmm.QMM_S32)):
        assert deq(**kw) == bad, kw

    def mm(a=P, ab=need, M=100, b=P, bb=need, N=100, K=200, bl=16, C=P, cd=F):
        return lib.qmm_fp4_matmul(a, ab, M, b, bb, N, K, bl, C, cd, None)
    for kw in (dict(a=None), dict(b=ODD), dict(ab=need - 1), dict(bb=0), dict(M=-1), dict(K=-1), dict(K=2 ** 31),
               dict(bl=17), dict(C=None), dict(cd=qmm.QMM_U8), dict(M=129)):
        assert mm(**kw) == bad, kw
    assert mm(M=0, a=None) == qmm.QMM_OK and mm(N=0, b=None) == qmm.QMM_OK


def test_python_refusals(qmm):
    """What the binding refuses before any pointer is taken (CPU tensors stand in)."""
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        qmm.qmm_rms_norm_s8(x, torch.ones(64))
    with pytest.raises(ValueError, match="CUDA"):
        qmm.qmm_rms_norm_backward(x, x, torch.ones(64), torch.ones(4))
    with pytest.raises(ValueError, match="CUDA"):
        qmm.qmm_fp4_quantize(x)
    m = qmm.Fp4Matrix(torch.zeros(1, dtype=torch.uint8), 4, 64, 16)
    with pytest.raises(ValueError, match="CUDA"):
        qmm.qmm_fp4_matmul(m, m)
    with pytest.raises(ValueError, match="CUDA"):
        qmm.qmm_fp4_dequantize(m)
