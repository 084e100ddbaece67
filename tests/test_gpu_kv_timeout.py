"""The bounded waits of attention for prompts, run on the GPU without any fault: a host-side test hook keeps the first
block of the kernel from copying its first keys. Its wait must run out after the short limit given, the error word
must name the site, the block must unwind (copies in flight, tensor memory) and return while the others finish, and
the next ordinary call must be right."""
import ctypes
import time

import pytest
import torch

from _kv import TYPES, Batch, rounded
from test_gpu_kv_attention import q  # noqa: F401
from test_kv_abi import Batch as CBatch
from test_kv_abi import Cache as CCache

pytestmark = pytest.mark.gpu

SITE_RAW = 0x503           # the converters' wait for int8 keys


def stalled(q, cache, table, lengths, starts, x, out, limit):  # noqa: F811
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    f = q.lib().qmm_test_kv_attention_stall
    f.argtypes = [vp, vp, vp, ctypes.c_int, i64, i64, i64, ctypes.c_float, ctypes.c_int, i64, vp, vp, ctypes.c_size_t,
                  ctypes.c_uint64, vp]
    f.restype = ctypes.c_int
    pages, heads, page, dim = cache.k.shape
    rows, batch = x.shape[0], len(lengths)
    ws = torch.empty(q.qmm_kv_attention_workspace_bytes(rows, batch, x.shape[1], heads, dim, x.dtype), dtype=torch.uint8,
                     device="cuda")
    c = CCache(*(t.data_ptr() for t in cache), pages, heads, page, dim)
    b = CBatch(table.data_ptr(), lengths.data_ptr(), starts.data_ptr(), batch, table.shape[1], rows)
    kind = q.QMM_F32 if x.dtype == torch.float32 else q.QMM_BF16
    return f(ctypes.byref(c), ctypes.byref(b), x.data_ptr(), kind, x.stride(0), x.stride(1), x.shape[1], dim ** -0.5, 1,
             rows, out.data_ptr(), ws.data_ptr(), ws.numel(), limit, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,length", [(400, 400), (100, 3000)])
def test_a_wait_that_runs_out(q, kind, dim, n, length):  # noqa: F811
    b = Batch([(n, length)], 2, dim, 64, seed=16)
    cache, table, lengths, starts = b.device(q)
    x = torch.from_numpy(rounded(b.rng.standard_normal((n, 8, dim)), kind)).to(TYPES[kind]).cuda()
    want = q.qmm_kv_attention(x, cache, table, lengths, starts=starts, max_tokens=n)
    lib, stream = q.lib(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.qmm_check_device_error(stream) == q.QMM_OK
    out = torch.full_like(x, 7)
    t0 = time.monotonic()
    assert stalled(q, cache, table, lengths, starts, x, out, 2_000_000) == q.QMM_OK
    # the kernel returns (the synchronisation inside the check ends), long before the ordinary limit, and says where
    assert lib.qmm_check_device_error(stream) == q.QMM_ERR_TIMEOUT
    assert time.monotonic() - t0 < 0.9
    assert lib.qmm_last_device_error() == SITE_RAW
    assert lib.qmm_check_device_error(stream) == q.QMM_OK
    # the block's rows are the first ones of the first key head; the last tokens and the other head are others'
    assert (out[0, 0] == 7).all()
    assert torch.equal(out[:, 4:], want[:, 4:])
    if n == length:
        assert torch.equal(out[64:], want[64:])
    assert torch.equal(q.qmm_kv_attention(x, cache, table, lengths, starts=starts, max_tokens=n), want)
    q.check_device_error()


def test_limits_outside_the_range_are_refused(q):  # noqa: F811
    x = torch.zeros(1, 1, 64, device="cuda")
    b = Batch([(1, 1)], 1, 64, 16).device(q)
    for limit in (0, 999, 100_000_001):
        assert stalled(q, *b, x, x, limit) == q.QMM_ERR_INVALID_ARG
