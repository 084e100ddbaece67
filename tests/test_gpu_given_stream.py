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


def check_owner(call, compare=True):
    """All memory that `call` allocates belongs to the stream it is given, and the values are those of
    the current stream's call."""
    want = call(None)
    torch.cuda.synchronize()   # (one call's outputs are host tensors)
    want = values(want)
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
    for a, b in zip(values(got), want) if compare else ():
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", LAYER)
def test_layer_calls_allocate_on_the_given_stream(name):
    check_owner(layer_calls()[name])


def check_neighbours(call, compare=True):
    """While the given stream is still busy, the current one allocates what the call let go of."""
    want = call(None)
    torch.cuda.synchronize()   # (one call's outputs are host tensors)
    want = values(want)
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
    for a, b in zip(values(got), want) if compare else ():
        assert torch.equal(a, b)
    del got
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", LAYER)
def test_layer_calls_beside_a_busy_current_stream(name):
    check_neighbours(layer_calls()[name])


def int8_calls():
    """The calls marshalled through ctypes."""
    g = torch.Generator(device="cuda").manual_seed(1)

    def ints(*n, lo=-128, t=torch.int8):
        return torch.randint(lo, lo + 256, n, generator=g, device="cuda", dtype=t)

    M, K, N = 512, 1024, 2048
    A, B, U = ints(M, K), ints(K, N), ints(M, K, lo=0, t=torch.uint8)
    sm, sn = (torch.rand(n, generator=g, device="cuda") for n in (M, N))
    x = torch.randn(M, K, generator=g, device="cuda")
    one = torch.rand(1, generator=g, device="cuda")
    xb, few = x.to(BF), x[:4].to(BF)
    packed, dqm = q.qmm_w8_pack_decode_weight(B), q.dynamic_quantize_matmul_pack_weight(B)
    img, ker = ints(2, 64, 28, 28), ints(64, 64, 3, 3)
    C = torch.empty(M, N, device="cuda")
    acc = torch.empty(M, N, dtype=torch.int32, device="cuda")
    hA, hB, hm, hn = (t.cpu().pin_memory() for t in (A, B, sm, sn))
    return {
        "a8w8": lambda s: (q.qmm_a8w8(A, B, sm, sn, stream=s),),
        # (the workspace alone is allocated)
        "a8w8_into": lambda s: (q.qmm_a8w8(A, B, sm, sn, out=C, stream=s),),
        "a8w8_acc": lambda s: (q.qmm_a8w8_acc(A, B, sm, sn, acc_out=acc, stream=s),),
        "a8w8_host": lambda s: (q.qmm_a8w8_host(hA, hB, hm, hn, stream=s),),
        "w8": lambda s: (q.qmm_w8_dequant(xb, B, sn, stream=s),),
        "w8_pack": lambda s: (q.qmm_w8_pack_decode_weight(B, stream=s),),
        "w8_packed": lambda s: (q.qmm_w8_dequant_packed(few, packed, N, sn, stream=s),),
        "matmul_integer": lambda s: (q.matmul_integer(U, B, stream=s),),
        "conv": lambda s: (q.conv_integer(img, ker, pads=[1, 1, 1, 1], stream=s),),
        "dql": lambda s: q.dynamic_quantize_linear(x, row_len=K, stream=s),
        "dqm": lambda s: q.dynamic_quantize_matmul(x, B, one, stream=s),
        "dqm_pack": lambda s: (q.dynamic_quantize_matmul_pack_weight(B, stream=s).buf,),
        "dqm_packed": lambda s: q.dynamic_quantize_matmul_packed(x, dqm, one, stream=s),
    }


INT8 = ["a8w8", "a8w8_into", "a8w8_acc", "a8w8_host", "w8", "w8_pack", "w8_packed", "matmul_integer", "conv", "dql",
        "dqm", "dqm_pack", "dqm_packed"]
# (their padding holds anything, and only the products made of them are compared)
PADDED = {"w8_pack", "dqm_pack"}


@pytest.mark.parametrize("name", INT8)
def test_int8_calls_allocate_on_the_given_stream(name):
    check_owner(int8_calls()[name], compare=name not in PADDED)


@pytest.mark.parametrize("name", INT8)
def test_int8_calls_beside_a_busy_current_stream(name):
    check_neighbours(int8_calls()[name], compare=name not in PADDED)
