"""Calls with stream=: they run on that stream, and what they allocate is that stream's
memory. Blocks of the caching allocator belong to the stream that allocated them; a
workspace from another stream's memory would be handed out again, on return, while
the kernels still use it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")

BF = torch.bfloat16
M, H, N = 700, 4096, 640


def layer_calls():
    """name -> call with a stream; the outputs of calls given their outputs are dropped."""
    g = torch.Generator(device="cuda").manual_seed(0)
    x, r, dy, dh = (torch.randn(M, H, generator=g, device="cuda").to(BF) for _ in range(4))
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF)
    b = torch.randn(N, H, generator=g, device="cuda").to(BF)
    n = q.qmm_rms_norm_s8(x, w, residual=r, save_rstd=True)
    a4, b4 = q.qmm_fp4_quantize(x), q.qmm_fp4_quantize(b)
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    return {
        "norm": lambda s: q.qmm_rms_norm_s8(x, w, residual=r, save_rstd=True, stream=s)[:],
        "read_s8": lambda s: (q.qmm_s8_dequantize_rows(n.q, n.scale, stream=s),),
        "grad": lambda s: q.qmm_rms_norm_backward(dy, n.h, w, n.rstd, dh=dh, stream=s),
        # (the workspace alone is allocated)
        "grad_into": lambda s: q.qmm_rms_norm_backward(dy, n.h, w, n.rstd, dh=dh, out=dx, dweight=dw, stream=s),
        "quantise": lambda s: (q.qmm_fp4_quantize(x, stream=s),),
        "quantise_t": lambda s: (q.qmm_fp4_quantize(x, transpose=True, stream=s),),
        "both": lambda s: q.qmm_fp4_quantize_both(x, stream=s),
        "read_fp4": lambda s: (q.qmm_fp4_dequantize(a4, stream=s),),
        "matmul": lambda s: (q.qmm_fp4_matmul(a4, b4, stream=s),),
    }


LAYER = ["norm", "read_s8", "grad", "grad_into", "quantise", "quantise_t", "both", "read_fp4", "matmul"]


def values(outputs):
    """Copies of the outputs, packed matrices read back (their padding holds anything)."""
    return [q.qmm_fp4_dequantize(t) if isinstance(t, q.Fp4Matrix) else t.clone() for t in outputs]


def check_owner(call):
    """All memory that `call` allocates belongs to the stream it is given, and the values are those of
    the current stream's call."""
    want = values(call(None))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    segments = torch.cuda.memory_snapshot
    mine = lambda es: sum(e["total_size"] for e in es if e["stream"] == s.cuda_stream)  # noqa: E731
    before = segments()
    torch.cuda.reset_peak_memory_stats()
    base = torch.cuda.memory_allocated()
    got = call(s)
    torch.cuda.synchronize()
    after = segments()
    assert torch.cuda.max_memory_allocated() > base          # (something was allocated)
    assert mine(after) > mine(before)
    assert sum(e["total_size"] for e in after) - mine(after) == sum(e["total_size"] for e in before) - mine(before)
    assert torch.cuda.current_stream() != s
    for a, b in zip(values(got), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", LAYER)
def test_layer_calls_allocate_on_the_given_stream(name):
    check_owner(layer_calls()[name])


def check_neighbours(call):
    """While the given stream is still busy, the current one allocates what the call let go of."""
    want = values(call(None))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)       # some 50 ms
    got = call(s)
    others = [torch.full((1 << k,), 7, dtype=torch.uint8, device="cuda") for k in range(9, 26) for _ in range(2)]
    torch.cuda.synchronize()
    for t in others:
        assert (t == 7).all()
    for a, b in zip(values(got), want):
        assert torch.equal(a, b)
    del got
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", LAYER)
def test_layer_calls_beside_a_busy_current_stream(name):
    check_neighbours(layer_calls()[name])
