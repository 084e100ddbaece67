"""Workloads of the operators around a quantised linear layer.

Five operators, each as its plain form (elementary torch operations in 32 bits)
and, where ``own`` is true, as the calls a user makes of this library:

  norm       h = x + residual;  RMS norm of h, quantised to int8 with one scale
             per row (what qmm_a8w8 takes as A and act_scale), read back
  norm_grad  the gradient of the norm (the quantiser passed straight through)
  quantise   a matrix to 4-bit floats with block scales, along its rows, along
             its columns, or both from one read, read back
  linear     y = x @ w.T on 4-bit operands: x quantised in the call, w kept
  train      one step of that layer: y, dx and dw, every operand quantised in
             the call, each along the axis its product sums over

4-bit floats are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, nearest,
ties to even). block 32: one power of two per 32 elements. block 16: one e4m3
scale per 16 elements and one float32 scale per row.
"""
import math

import torch

own = False

C127 = 127.0
R2688 = 1.0 / 2688.0      # 6 * 448: largest e2m1 times largest e4m3
R6 = 1.0 / 6.0
TINY = 2.0 ** -100        # a row scale below this stores the row as zeros
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # decoding one token of a 4096-wide model: the call's latency is all there is
        dict(name="norm_token", op="norm", rows=1, cols=4096, type="bf16", residual=True),
        # a prompt's worth of rows, the width and rows of this library's DynamicQuantizeLinear benchmark
        dict(name="norm_prompt", op="norm", rows=8192, cols=4096, type="bf16", residual=True),
        # float32 activations, an odd width (no vector loads), no residual
        dict(name="norm_odd_f32", op="norm", rows=1009, cols=5003, type="f32", residual=False),
        # training: the norm's gradient for a batch of 4096 tokens, with the gradient of the residual path
        dict(name="norm_grad_batch", op="norm_grad", rows=4096, cols=4096, type="bf16", residual=True),
        # a wide layer's ragged batch in float32, no residual path
        dict(name="norm_grad_wide_f32", op="norm_grad", rows=1531, cols=11008, type="f32", residual=False),
        # a decoding batch's activations: a few rows, latency
        dict(name="quantise_batch_rows", op="quantise", rows=16, cols=8192, type="bf16", block=16, axis="rows"),
        # a training batch's activations for the forward product and the weight's gradient, one read
        dict(name="quantise_both", op="quantise", rows=8192, cols=4096, type="bf16", block=32, axis="both"),
        # float32 master weights with ragged edges, along the columns
        dict(name="quantise_cols_odd_f32", op="quantise", rows=4099, cols=1021, type="f32", block=16, axis="cols"),
        # decoding one token: the shape of this library's decode benchmark; the weight's bytes are all there is
        dict(name="linear_token", op="linear", rows=1, inner=8192, cols=28672, type="bf16", block=16, out="bf16"),
        # a ragged decoding batch, an inner length that ends inside a block
        dict(name="linear_batch_odd", op="linear", rows=137, inner=4100, cols=11007, type="bf16", block=32, out="f32"),
        # a prompt: the product of this library's MatMulInteger benchmark
        dict(name="linear_prompt", op="linear", rows=8192, inner=4096, cols=11008, type="bf16", block=16, out="bf16"),
        # one training step of a layer, batch of 4096 tokens
        dict(name="train_step", op="train", rows=4096, inner=4096, cols=11008, type="bf16", block=32, out="bf16"),
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; half of the draws rounded to a multiple of 64 where that is possible."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 128 and rng.random() < 0.5:
        v = v // 64 * 64
    if v == 3072:
        v = 3073
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantise", "linear", "linear", "train"])
    kind = "bf16" if rng.random() < 0.7 else "f32"
    if op in ("norm", "norm_grad"):
        return dict(op=op, rows=_size(rng, 1, 8192), cols=_size(rng, 64, 16384), type=kind,
                    residual=rng.random() < 0.6)
    if op == "quantise":
        return dict(op=op, rows=_size(rng, 1, 8192), cols=_size(rng, 32, 16384), type=kind,
                    block=rng.choice([16, 32]), axis=rng.choice(["rows", "cols", "both"]))
    if op == "linear":
        inner, cols = _size(rng, 128, 8192), _size(rng, 64, 11008)
        rows = _size(rng, 1, min(8192, 360_000_000_000 // (inner * cols)))   # no more than linear_prompt
        return dict(op=op, rows=rows, inner=inner, cols=cols, type=kind, block=rng.choice([16, 32]),
                    out=rng.choice(["bf16", "f32"]))
    return dict(op=op, rows=_size(rng, 64, 4096), inner=_size(rng, 64, 4096), cols=_size(rng, 64, 8192), type=kind,
                block=rng.choice([16, 32]), out=rng.choice(["bf16", "f32"]))


def _inputs(case, seed):
    """The case's tensors: activations with a few large channels and rare outliers, weights of a linear layer."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    t = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def activations(rows, cols):
        x = normal(rows, cols)
        x *= 1.0 + 19.0 * (uniform(cols) < 0.004)
        x *= torch.where(uniform(rows, cols) < 0.001, 20.0, 1.0)
        return x.to(t)

    op, s = case["op"], {"case": dict(case)}
    if op == "norm":
        s["x"] = activations(case["rows"], case["cols"])
        s["residual"] = (2.0 * activations(case["rows"], case["cols"]).float()).to(t) if case["residual"] else None
        s["weight"] = (1.0 + 0.1 * normal(case["cols"])).to(t)
    elif op == "norm_grad":
        s["h"] = activations(case["rows"], case["cols"])
        s["weight"] = (1.0 + 0.1 * normal(case["cols"])).to(t)
        s["dy"] = (0.01 * normal(case["rows"], case["cols"])).to(t)
        s["dh"] = (0.01 * normal(case["rows"], case["cols"])).to(t) if case["residual"] else None
        hf = s["h"].float()
        s["rstd"] = torch.rsqrt((hf * hf).mean(dim=1) + 1e-6)   # kept from the forward pass
    elif op == "quantise":
        s["x"] = activations(case["rows"], case["cols"])
    else:
        s["x"] = activations(case["rows"], case["inner"])
        s["w"] = (normal(case["cols"], case["inner"]) / math.sqrt(case["inner"])).to(t)
        if op == "train":
            s["dy"] = (0.01 * normal(case["rows"], case["cols"])).to(t)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "linear":
        # a server quantises its weight once and keeps only that: here the library's packed form, or
        # the plain form's 4-bit codes (two to a byte), scale bytes and row scales
        w = s.pop("w")
        if own:
            import quantized_int8_matmul_gb300 as q
            s["w"] = q.qmm_fp4_quantize(w, block=case["block"])
        else:
            codes, scales, rowscale = _quantise(w.float(), case["block"])
            s["w"] = ((codes[:, 0::2] | (codes[:, 1::2] << 4)), scales, rowscale)
    return s


def work(case):
    e = 2 if case["type"] == "bf16" else 4
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["cols"]
        # x (and the residual) in; the sum, the int8 values as read back, the row scales out
        return {"bytes": n * (2 * e + (2 * e if case["residual"] else 0)) + 4 * case["rows"] + e * case["cols"],
                "flops": 6 * n}
    if op == "norm_grad":
        n = case["rows"] * case["cols"]
        return {"bytes": n * e * (3 + (1 if case["residual"] else 0)) + 4 * case["rows"] + (e + 4) * case["cols"],
                "flops": 10 * n}
    if op == "quantise":
        n = case["rows"] * case["cols"]
        return {"bytes": n * e * (3 if case["axis"] == "both" else 2), "flops": 4 * n}
    m, k, n, b = case["rows"], case["inner"], case["cols"], case["block"]
    o = 2 if case["out"] == "bf16" else 4
    if op == "linear":
        return {"bytes": m * k * e + n * k * (0.5 + 1.0 / b) + (4 * n if b == 16 else 0) + m * n * o,
                "flops": 2 * m * n * k}
    return {"bytes": e * (m * k + n * k + m * n) + o * (m * n + m * k) + 4 * n * k, "flops": 6 * m * n * k}


# ---------------------------------------------------------------------------
# The plain form
# ---------------------------------------------------------------------------
def _pad(x, block):
    """Columns padded with zeros to whole blocks."""
    r = -x.shape[1] % block
    return torch.cat([x, x.new_zeros(x.shape[0], r)], dim=1) if r else x


def _codes(v):
    """e2m1 codes of v: nearest, ties to the even code, beyond 6 to 6; the sign in bit 3."""
    m = v.abs()
    c = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    return c | (torch.signbit(v).to(torch.uint8) << 3)


def _quantise(x, block):
    """(codes [rows, padded], scale bytes [rows, blocks], row scales [rows] or None) of float32 x."""
    x = _pad(x, block)
    rows, cols = x.shape
    b = x.view(rows, cols // block, block)
    bmax = b.abs().amax(dim=2)
    if block == 32:
        byte = ((bmax.view(torch.int32) >> 23) - 2).clamp(min=0)
        up = ((254 - byte) << 23).view(torch.float32)      # 2^-(byte - 127)
        return _codes(b * up[:, :, None]).view(rows, cols), byte.to(torch.uint8), None
    g = bmax.amax(dim=1) * R2688
    g = torch.where(g < TINY, 1.0, g)
    u = torch.ones_like(g) / g
    s8 = ((bmax * u[:, None]) * R6).to(torch.float8_e4m3fn)
    s = s8.float()
    inv = torch.where(s > 0, u[:, None] / s, 0.0)
    return _codes(b * inv[:, :, None]).view(rows, cols), s8.view(torch.uint8), g


def _values(codes, scales, block):
    """code value x block scale, in float32 (the row scale is not in it)."""
    lut = torch.tensor([*E2M1, *(-v for v in E2M1)], device=codes.device)
    e = lut[codes.int()]
    if block == 32:
        i = scales.to(torch.int32)
        s = torch.where(i == 0, 2.0 ** -127, (i.clamp(min=1) << 23).view(torch.float32))
    else:
        s = scales.view(torch.float8_e4m3fn).float()
    rows, cols = codes.shape
    return (e.view(rows, cols // block, block) * s[:, :, None]).view(rows, cols)


def _read_back(x, block, dtype):
    c, s, g = _quantise(x, block)
    v = _values(c, s, block)[:, :x.shape[1]]
    return (v if g is None else v * g[:, None]).to(dtype)


def _product(a, b, block, dtype):
    (ca, sa, ga), (cb, sb, gb) = a, b
    y = _values(ca, sa, block) @ _values(cb, sb, block).T
    if ga is not None:
        y = (y * ga[:, None]) * gb[None, :]
    return y.to(dtype)


def _run_plain(state):
    case = state["case"]
    op, t = case["op"], TYPES[case["type"]]
    if op == "norm":
        h = state["x"]
        if state["residual"] is not None:
            h = (h.float() + state["residual"].float()).to(t)
        hf = h.float()
        rstd = torch.rsqrt((hf * hf).mean(dim=1) + 1e-6)
        v = hf * state["weight"].float()
        amax = v.abs().amax(dim=1)
        inv = torch.full_like(amax, C127) / amax
        inv = torch.where(amax > 0, inv, 0.0)
        scale = torch.where(amax > 0, (amax * rstd) * (1.0 / 127.0), 1.0)
        q = torch.round(v * inv[:, None]).clamp(-127, 127).to(torch.int8)
        out = {"values": (q.float() * scale[:, None]).to(t), "scale": scale}
        if state["residual"] is not None:
            out["h"] = h
        return out
    if op == "norm_grad":
        h, w, dy, rstd = state["h"].float(), state["weight"].float(), state["dy"].float(), state["rstd"]
        n = h * rstd[:, None]
        g = dy * w
        dx = (g - n * (g * n).mean(dim=1, keepdim=True)) * rstd[:, None]
        if state["dh"] is not None:
            dx = dx + state["dh"].float()
        return {"dx": dx.to(t), "dweight": (dy * n).sum(dim=0)}
    block = case["block"]
    if op == "quantise":
        x = state["x"].float()
        out = {}
        if case["axis"] in ("rows", "both"):
            out["rows"] = _read_back(x, block, t)
        if case["axis"] in ("cols", "both"):
            out["cols"] = _read_back(x.T.contiguous(), block, t)
        return out
    o = TYPES[case["out"]]
    x = state["x"].float()
    if op == "linear":
        packed, scales, rowscale = state["w"]
        codes = torch.stack([packed & 15, packed >> 4], dim=2).view(packed.shape[0], -1)
        return _product(_quantise(x, block), (codes, scales, rowscale), block, o)
    w, dy = state["w"].float(), state["dy"].float()
    xt, wt, dyt = (v.T.contiguous() for v in (x, w, dy))
    return {"y": _product(_quantise(x, block), _quantise(w, block), block, o),
            "dx": _product(_quantise(dy, block), _quantise(wt, block), block, o),
            "dw": _product(_quantise(dyt, block), _quantise(xt, block), block, torch.float32)}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _run_own(state):
    import quantized_int8_matmul_gb300 as q
    case = state["case"]
    op, t = case["op"], TYPES[case["type"]]
    if op == "norm":
        r = q.qmm_rms_norm_s8(state["x"], state["weight"], residual=state["residual"], eps=1e-6)
        out = {"values": q.qmm_s8_dequantize_rows(r.q, r.scale, out_dtype=t), "scale": r.scale}
        if state["residual"] is not None:
            out["h"] = r.h
        return out
    if op == "norm_grad":
        dx, dw = q.qmm_rms_norm_backward(state["dy"], state["h"], state["weight"], state["rstd"], dh=state["dh"])
        return {"dx": dx, "dweight": dw}
    block = case["block"]
    if op == "quantise":
        x, axis = state["x"], case["axis"]
        if axis == "both":
            r, c = q.qmm_fp4_quantize_both(x, block=block)
            return {"rows": q.qmm_fp4_dequantize(r, out_dtype=t), "cols": q.qmm_fp4_dequantize(c, out_dtype=t)}
        return {axis: q.qmm_fp4_dequantize(q.qmm_fp4_quantize(x, block=block, transpose=axis == "cols"),
                                           out_dtype=t)}
    o = TYPES[case["out"]]
    if op == "linear":
        return q.qmm_fp4_matmul(q.qmm_fp4_quantize(state["x"], block=block), state["w"], out_dtype=o)
    x, xt = q.qmm_fp4_quantize_both(state["x"], block=block)
    w, wt = q.qmm_fp4_quantize_both(state["w"], block=block)
    y = q.qmm_fp4_matmul(x, w, out_dtype=o)
    dy, dyt = q.qmm_fp4_quantize_both(state["dy"], block=block)
    return {"y": y, "dx": q.qmm_fp4_matmul(dy, wt, out_dtype=o),
            "dw": q.qmm_fp4_matmul(dyt, xt, out_dtype=torch.float32)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_fp4(x, block):
    """The values that float64 x stands for once stored in 4 bits with block scales."""
    rows, cols = x.shape
    pad = -cols % block
    x = torch.nn.functional.pad(x, (0, pad)).reshape(rows, -1, block)
    top = x.abs().max(dim=2, keepdim=True).values
    if block == 32:
        _, e = torch.frexp(top)                      # top in [2^(e-1), 2^e)
        s = torch.ldexp(torch.ones_like(top), (e - 3).clamp(min=-127))
    else:
        g = top.max(dim=1, keepdim=True).values / 2688.0
        g[g < TINY] = 1.0
        t = top / g / 6.0
        _, e = torch.frexp(t)
        step = torch.ldexp(torch.ones_like(t), (e - 1).clamp(min=-6) - 3)
        s = torch.minimum(torch.round(t / step) * step, torch.full_like(t, 448.0)) * g
    m = torch.where(s > 0, x.abs() / s.clamp(min=1e-300), torch.zeros_like(x))
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).to(m.dtype)
    r = (torch.round(m / step) * step).clamp(max=6.0)
    return (torch.copysign(r, x) * s).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    s = _inputs(case, seed)
    op, t = case["op"], TYPES[case["type"]]
    if op == "norm":
        h = s["x"]
        if case["residual"]:
            h = (s["x"].double() + s["residual"].double()).float().to(t)   # the sum is kept in the inputs' type
        d = h.double()
        rms = ((d ** 2).sum(1) / d.shape[1] + 1e-6).sqrt()
        v = d * s["weight"].double()
        top = v.abs().max(1).values
        scale = torch.where(top > 0, top / rms / 127.0, torch.ones_like(top))
        q = torch.round(v * 127.0 / top.clamp(min=1e-300)[:, None])
        out = {"values": q * scale[:, None], "scale": scale}
        if case["residual"]:
            out["h"] = d
        return out
    if op == "norm_grad":
        h, w, dy, r = s["h"].double(), s["weight"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        wdy = w * dy
        dx = r * wdy - h * r ** 3 * (wdy * h).sum(1, keepdim=True) / h.shape[1]
        if case["residual"]:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dweight": (dy * h * r).sum(0)}
    block, x = case["block"], s["x"].double()
    if op == "quantise":
        out = {}
        if case["axis"] != "cols":
            out["rows"] = _exact_fp4(x, block)
        if case["axis"] != "rows":
            out["cols"] = _exact_fp4(x.T, block)
        return out
    w = s["w"].double()
    y = _exact_fp4(x, block) @ _exact_fp4(w, block).T
    if op == "linear":
        return y
    dy = s["dy"].double()
    return {"y": y, "dx": _exact_fp4(dy, block) @ _exact_fp4(w.T, block).T,
            "dw": _exact_fp4(dy.T, block) @ _exact_fp4(x.T, block).T}
