"""Extents at the ends of what the norm's and the 4-bit entry points take, on the host,
without a GPU: what is refused before anything is launched."""
import ctypes

import pytest

P = ctypes.c_void_p(256)
MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def qmm():
    import quantized_int8_matmul_gb300 as q
    lib = q.lib()
    i64, vp, ci, sz, cf = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    lib.qmm_rms_norm_s8.argtypes = [vp, ci, i64, i64, i64, vp, i64, vp, ci, cf, vp, vp, vp, vp, vp]
    lib.qmm_rms_norm_backward.argtypes = [vp, i64, vp, i64, vp, i64, ci, i64, i64, vp, ci, vp, vp, vp, vp, sz, vp]
    return q


@pytest.mark.parametrize("H", [MAX, MAX - 8191, MAX - 2 ** 14 + 1])
def test_norm_rows_too_wide_for_32_bit_indexes_are_refused(qmm, H):
    """A CTA's last vectors reach past H by up to 8 * 1024 elements: not past 2^31."""
    lib, F, no = qmm.lib(), qmm.QMM_F32, qmm.QMM_ERR_UNSUPPORTED
    for t in (F, qmm.QMM_BF16):
        assert lib.qmm_rms_norm_s8(P, t, 1, H, H, None, 0, P, t, 1e-6, None, P, P, None, None) == no
        assert lib.qmm_rms_norm_backward(P, H, P, H, None, 0, t, 1, H, P, t, P, ctypes.c_void_p(512), P, P, 2 ** 40,
                                         None) == no
        assert lib.qmm_rms_norm_backward(P, H, P, H, None, 0, t, 0, H, P, t, P, ctypes.c_void_p(512), P, P, 2 ** 40,
                                         None) == no
    assert qmm.qmm_rms_norm_backward_workspace_bytes(1, H) == 0
    assert qmm.qmm_rms_norm_backward_workspace_bytes(1, MAX - 2 ** 14) == 4 * (MAX - 2 ** 14)
