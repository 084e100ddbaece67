"""The native marshalling of the norm's and the 4-bit calls on a host without a GPU:
what it raises for tensors that have no memory behind them. Fake CUDA tensors
(extents, type and device, no storage) stand in for real ones. What could end the
process runs in one of its own."""
import os
import subprocess
import sys
import textwrap

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PRELUDE = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import quantized_int8_matmul_gb300 as q

class Stream:
    cuda_stream = 0

S, F32, U8, S8 = Stream(), torch.float32, torch.uint8, torch.int8

def outcome(f, *a):
    try:
        f(*a)
        return "returned"
    except Exception as e:
        return type(e).__name__ + ": " + str(e)

def fake(*shape, dtype=F32, device="cuda:0"):
    return torch.empty(*shape, dtype=dtype, device=device)
"""


def child(body):
    """The lines that `body` prints, run under fake tensors in a process of its own."""
    code = PRELUDE + "with FakeTensorMode(allow_non_fake_inputs=True):\n" + textwrap.indent(textwrap.dedent(body), "    ")
    env = {**os.environ, "CUDA_VISIBLE_DEVICES": ""}   # (with a GPU in sight, fake tensors are on real devices only)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, f"exit code {r.returncode}\n{r.stdout}\n{r.stderr[-2000:]}"
    return r.stdout.splitlines()


def test_batched_tensors_raise():
    """Inside torch.vmap a tensor has no pointer of its own: an error, as the ctypes calls give, not the
    end of the process."""
    lines = child("""
    B, M, N, H = 3, 4, 5, 128
    rows, scale = fake(B, M, H, dtype=S8), fake(B, M)
    x, y, w, dw = fake(B, M, H), fake(B, M, H), fake(H), fake(B, H)
    ws = fake(q.qmm_rms_norm_backward_workspace_bytes(M, H), dtype=U8)
    p = fake(B, q.qmm_fp4_bytes(M, H, 16), dtype=U8)
    pt, pn = fake(B, q.qmm_fp4_bytes(H, M, 16), dtype=U8), fake(q.qmm_fp4_bytes(N, H, 16), dtype=U8)
    C = fake(B, M, N)
    mat = lambda b, r=M, c=H: q.Fp4Matrix(b, r, c, 16)
    calls = {
        "s8": (lambda a, s, o: q.qmm_s8_dequantize_rows(a, s, out=o, out_dtype=F32, stream=S), rows, scale, y),
        "grad": (lambda d, h, r, o, g: q.qmm_rms_norm_backward(d, h, w, r, out=o, dweight=g, stream=S, workspace=ws),
                 x, x, scale, y, dw),
        "quantise": (lambda t, o: q.qmm_fp4_quantize(t, out=mat(o), stream=S), x, p),
        "both": (lambda t, o, r: q.qmm_fp4_quantize_both(t, out=mat(o), out_t=mat(r, H, M), stream=S), x, p, pt),
        "read": (lambda b, o: q.qmm_fp4_dequantize(mat(b), out=o, out_dtype=F32, stream=S), p, y),
        "matmul": (lambda b, o: q.qmm_fp4_matmul(mat(b), mat(pn, N), out=o, out_dtype=F32, stream=S), p, C),
        "norm": (lambda t, o: q.qmm_rms_norm_s8(t, w, out=o, stream=S), x, rows),
    }
    for name, (f, *args) in calls.items():
        print(name, outcome(torch.vmap(f), *args))
    """)
    assert len(lines) == 7
    for line in lines:
        assert line.split()[1] == "RuntimeError:", line
    for line in lines[:6]:   # (the norm allocates its scales first, which fails without a GPU)
        assert "data pointer" in line, line


def test_errors_inside_arguments_are_raised():
    """A truth value that raises is that error, not a result with an error pending; a block that is no
    int is refused, not cut to its low bits."""
    lines = child("""
    class Bad:
        def __bool__(self):
            raise ZeroDivisionError("no truth value")

    x, w = fake(4, 64), fake(64)
    print(outcome(lambda: q.qmm_rms_norm_s8(x, w, save_rstd=Bad(), stream=S)))
    m = q.Fp4Matrix(fake(q.qmm_fp4_bytes(4, 64, 16), dtype=U8), 4, 64, 2 ** 32 + 16)
    print(outcome(lambda: q.qmm_fp4_dequantize(m, out=x, out_dtype=F32, stream=S)))
    print(outcome(lambda: q.qmm_fp4_matmul(m, m, out=fake(4, 4), out_dtype=F32, stream=S)))
    print(outcome(lambda: q.qmm_fp4_quantize(x, block=2 ** 32 + 16, stream=S)))
    """)
    assert lines[0] == "ZeroDivisionError: no truth value"
    assert len(lines) == 4 and all(line == "ValueError: block must be 16 or 32" for line in lines[1:]), lines


def test_operands_on_two_devices_are_refused():
    lines = child("""
    M, N, H = 4, 5, 64
    a, b = (lambda *s, **k: fake(*s, device="cuda:0", **k)), (lambda *s, **k: fake(*s, device="cuda:1", **k))
    x, w, rows, scale = a(M, H), a(H), a(M, H, dtype=S8), a(M)
    p = q.Fp4Matrix(a(q.qmm_fp4_bytes(M, H, 16), dtype=U8), M, H, 16)
    far = q.Fp4Matrix(b(q.qmm_fp4_bytes(N, H, 16), dtype=U8), N, H, 16)
    ws = a(q.qmm_rms_norm_backward_workspace_bytes(M, H), dtype=U8)
    calls = [
        lambda: q.qmm_rms_norm_s8(x, b(H), stream=S),
        lambda: q.qmm_rms_norm_s8(x, w, residual=b(M, H), stream=S),
        lambda: q.qmm_rms_norm_s8(x, w, out=b(M, H, dtype=S8), stream=S),
        lambda: q.qmm_s8_dequantize_rows(rows, b(M), stream=S),
        lambda: q.qmm_s8_dequantize_rows(rows, scale, out=b(M, H), stream=S),
        lambda: q.qmm_rms_norm_backward(b(M, H), x, w, scale, stream=S),
        lambda: q.qmm_rms_norm_backward(x, x, b(H), scale, stream=S),
        lambda: q.qmm_rms_norm_backward(x, x, w, b(M), stream=S),
        lambda: q.qmm_rms_norm_backward(x, x, w, scale, dh=b(M, H), stream=S),
        lambda: q.qmm_rms_norm_backward(x, x, w, scale, out=b(M, H), dweight=a(H), workspace=ws, stream=S),
        lambda: q.qmm_rms_norm_backward(x, x, w, scale, out=a(M, H), dweight=b(H), workspace=ws, stream=S),
        lambda: q.qmm_rms_norm_backward(x, x, w, scale, out=a(M, H), dweight=a(H), stream=S,
                                        workspace=b(ws.numel(), dtype=U8)),
        lambda: q.qmm_fp4_quantize(x, out=q.Fp4Matrix(b(p.buf.numel(), dtype=U8), M, H, 16), stream=S),
        lambda: q.qmm_fp4_dequantize(p, out=b(M, H), stream=S),
        lambda: q.qmm_fp4_matmul(p, far, stream=S),
        lambda: q.qmm_fp4_matmul(p, p, out=b(M, M), stream=S),
    ]
    for f in calls:
        print(outcome(f))
    """)
    assert len(lines) == 16
    for i, line in enumerate(lines):
        assert line.startswith("ValueError: ") and "cuda:1" in line and "cuda:0" in line, (i, line)


def test_int8_operands_off_the_current_device_are_refused():
    lines = child("""
    torch._C._cuda_getDevice = lambda: 0        # (there is no driver to ask)
    far = lambda *s, **k: fake(*s, device="cuda:1", **k)
    A, B, near = fake(4, 64, dtype=S8), fake(64, 32, dtype=S8), fake(1)
    x = fake(4, 64)
    calls = [
        lambda: q.qmm_a8w8(far(4, 64, dtype=S8), B, near, near, stream=S),
        lambda: q.qmm_a8w8(A, B, near, far(1), stream=S),
        lambda: q.qmm_a8w8(A, B, near, near, out=far(4, 32), stream=S),
        lambda: q.qmm_a8w8_acc(A, far(64, 32, dtype=S8), near, near, stream=S),
        lambda: q.qmm_w8_dequant(x, B, far(1), stream=S),
        lambda: q.matmul_integer(A, far(64, 32, dtype=S8), stream=S),
        lambda: q.dynamic_quantize_linear(far(4, 64), stream=S),
        lambda: q.dynamic_quantize_matmul(x, far(64, 32, dtype=S8), near, stream=S),
    ]
    for f in calls:
        print(outcome(f))
    """)
    assert len(lines) == 8
    for i, line in enumerate(lines):
        assert line.startswith("ValueError: ") and "cuda:1" in line and "cuda:0" in line, (i, line)


def test_a_workspace_that_repeats_its_memory_is_refused():
    """An expanded tensor has fewer bytes behind it than elements."""
    lines = child("""
    x, w, r = fake(4, 64), fake(64), fake(4)
    n = q.qmm_rms_norm_backward_workspace_bytes(4, 64)
    for ws in (fake(1, dtype=U8).expand(n), torch.empty_strided((n,), (2,), dtype=U8, device="cuda:0")):
        print(outcome(lambda: q.qmm_rms_norm_backward(x, x, w, r, out=fake(4, 64), dweight=fake(64), stream=S,
                                                      workspace=ws)))
    """)
    assert lines == ["ValueError: workspace must be contiguous"] * 2, lines
