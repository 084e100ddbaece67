"""Nothing is written outside the outputs and workspaces of the norm's and the 4-bit
calls: each lies between guard bytes, which stay as they are, at widths and offsets off
every vector and tile boundary."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 512


class Guards:
    """Tensors cut out of buffers of 0xA5; off: elements past a 512-byte boundary."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype, off=0):
        size = torch.empty(0, dtype=dtype).element_size()
        n = 1
        for d in shape:
            n *= d
        raw = torch.full((2 * GUARD + (n + off) * size,), 0xA5, dtype=torch.uint8, device="cuda")
        beg = GUARD + off * size
        self.all.append((raw, beg, beg + n * size))
        return raw[beg:beg + n * size].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for i, (raw, beg, end) in enumerate(self.all):
            assert (raw[:beg] == 0xA5).all() and (raw[end:] == 0xA5).all(), f"buffer {i}"


def randn(*shape, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


ROWS = [(1, 1), (3, 7), (5, 33), (2, 64), (7, 1001), (33, 4096), (9, 5003), (2, 40001), (700, 251), (401, 4099),
        (320, 1024), (1500, 4101)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("M,H", ROWS)
def test_norm(M, H, off, dt):
    t, G = TYPES[dt], Guards()
    x, r, w = randn(M, H, dt=t), randn(M, H, dt=t, seed=1), randn(H, dt=t, seed=2)
    lib = q.lib()
    i64, vp, ci, cf = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.qmm_rms_norm_s8.argtypes = [vp, ci, i64, i64, i64, vp, i64, vp, ci, cf, vp, vp, vp, vp, vp]
    ty = q.QMM_BF16 if dt == "bf16" else q.QMM_F32
    s = torch.cuda.current_stream().cuda_stream
    for res in (True, False):
        h, o, sc, rs = G((M, H), t, off), G((M, H), torch.int8, off), G((M,), torch.float32), G((M,), torch.float32)
        assert lib.qmm_rms_norm_s8(x.data_ptr(), ty, M, H, H, r.data_ptr() if res else None, H, w.data_ptr(), ty, 1e-6,
                                   h.data_ptr(), o.data_ptr(), sc.data_ptr(), rs.data_ptr(), s) == q.QMM_OK
        want = q.qmm_rms_norm_s8(x, w, residual=r if res else None, save_rstd=True)
        assert torch.equal(o, want.q) and torch.equal(h, want.h)
        for y in (torch.float32, torch.bfloat16):
            q.qmm_s8_dequantize_rows(o, sc, out=G((M, H), y, off))
        ws = G((q.qmm_rms_norm_backward_workspace_bytes(M, H),), torch.uint8)
        q.qmm_rms_norm_backward(r, h, w, rs, dh=x if res else None, out=G((M, H), t, off),
                                dweight=G((H,), torch.float32, off), workspace=ws)
    q.check_device_error()
    G.check()


MATS = [(1, 1), (1, 33), (3, 130), (16, 4100), (129, 127), (257, 515), (1024, 200), (1025, 333), (1300, 8208), (2, 20001)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", MATS)
def test_fp4(R, C, dt, block):
    G = Guards()
    x = randn(R, C, dt=TYPES[dt])

    def packed(rows, cols):
        return q.Fp4Matrix(G((q.qmm_fp4_bytes(rows, cols, block),), torch.uint8), rows, cols, block)

    a = q.qmm_fp4_quantize(x, block=block, out=packed(R, C))
    b = q.qmm_fp4_quantize(x, block=block, transpose=True, out=packed(C, R))
    c, d = q.qmm_fp4_quantize_both(x, block=block, out=packed(R, C), out_t=packed(C, R))
    for y in (torch.float32, torch.bfloat16):
        for off in (0, 1):
            for m in (a, b, c, d):
                q.qmm_fp4_dequantize(m, out=G((m.rows, m.cols), y, off), out_dtype=y)
    q.check_device_error()
    G.check()


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 33, 100), (3, 1000, 513), (16, 129, 4100), (64, 300, 128),
                                   (65, 129, 640), (100, 65, 300), (137, 1003, 257), (256, 257, 512), (300, 1024, 129),
                                   (520, 77, 1000), (1500, 3001, 260)])
def test_products(M, N, K, block):
    G = Guards()
    a, b = (q.qmm_fp4_quantize(randn(n, K, dt=torch.bfloat16, seed=n), block=block) for n in (M, N))
    for y in (torch.float32, torch.bfloat16):
        want = q.qmm_fp4_matmul(a, b, out_dtype=y)
        for off in (0, 1, 2):
            assert torch.equal(q.qmm_fp4_matmul(a, b, out=G((M, N), y, off), out_dtype=y), want)
    q.check_device_error()
    G.check()
