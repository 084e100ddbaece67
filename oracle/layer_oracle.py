"""Plain numpy definitions of the operators around a quantised linear layer: the
RMS norm to int8 rows and its gradient, 4-bit floats with block scales, and
their product. Test infrastructure; shares no code with the CUDA path.

The integers and codes are decided by float32 steps that the definition fixes
one rounding at a time (numpy float32 arithmetic); sums, products and gradients
are float64."""
import numpy as np

F = np.float32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TINY = F(2.0 ** -100)


def bf16_round(x):
    """Round float32 to the nearest bfloat16 value (ties to even), as float32."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    b = x.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), r, x)


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------
def rms_norm_s8(x, w, residual, eps, bf16):
    """(q int8, scale float64, h float32, rstd float64) of float32 x, w."""
    with np.errstate(all="ignore"):
        h = x.astype(F)
        if residual is not None:
            h = h + residual.astype(F)
            h = bf16_round(h) if bf16 else h
        v = h * w.astype(F)
        a = np.abs(v).max(axis=1)
        bad = ~np.isfinite(v).all(axis=1)
        inv = np.where((a >= TINY) & ~bad, F(127) / np.where(a >= TINY, a, F(1)), F(0)).astype(F)
        p = np.clip((v * inv[:, None]).astype(F), F(-127), F(127))
        q = np.where(bad[:, None], 0, np.rint(np.where(bad[:, None], 0, p))).astype(np.int8)
        rstd = 1.0 / np.sqrt((h.astype(np.float64) ** 2).mean(axis=1) + eps)
        scale = np.where(bad, np.nan, np.where(a >= TINY, a.astype(np.float64) * rstd / 127.0, 1.0))
    return q, scale, h, rstd


def rms_norm(h, w, eps):
    """The normalised rows in float64 (what q * scale stands for)."""
    h = h.astype(np.float64)
    return h / np.sqrt((h ** 2).mean(axis=1, keepdims=True) + eps) * w.astype(np.float64)


def rms_norm_backward(dy, h, w, rstd, dh=None):
    """(dx, dweight) in float64 from the given rstd."""
    dy, h, w = (np.asarray(t, dtype=np.float64) for t in (dy, h, w))
    n = h * np.asarray(rstd, dtype=np.float64)[:, None]
    g = dy * w
    dx = (g - n * (g * n).mean(axis=1, keepdims=True)) * np.asarray(rstd, dtype=np.float64)[:, None]
    if dh is not None:
        dx = dx + np.asarray(dh, dtype=np.float64)
    return dx, (dy * n).sum(axis=0)


# ---------------------------------------------------------------------------
# 4-bit floats with block scales
# ---------------------------------------------------------------------------
def e2m1(v):
    """The nearest of +-E2M1, ties to the even code, beyond 6 to 6 (float64 values)."""
    m = np.minimum(np.abs(v.astype(np.float64)), 6.0)
    d = np.abs(m[..., None] - E2M1)
    lo = d.argmin(axis=-1)                       # the first of two equally near: the smaller code
    hi = np.minimum(lo + 1, 7)
    tie = np.take_along_axis(d, lo[..., None], -1) == np.take_along_axis(d, hi[..., None], -1)
    code = np.where(tie[..., 0] & (lo % 2 == 1), hi, lo)
    return np.copysign(E2M1[code], v)


E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])   # code 127 is NaN


def e4m3(v):
    """The nearest non-negative e4m3 value, ties to the even code, beyond 448 to 448."""
    v = np.minimum(v.astype(np.float64), 448.0)
    hi = np.clip(np.searchsorted(E4M3, v), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = v - E4M3[lo], E4M3[hi] - v
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, E4M3[hi], E4M3[lo])


def fp4(x, block):
    """(values without the row scale float64 [R, C], row scales float64 [R]) of float32 x."""
    x = np.asarray(x, dtype=F)
    R, C = x.shape
    xb = np.pad(x, ((0, 0), (0, -C % block))).reshape(R, -1, block)
    with np.errstate(all="ignore"):
        b = np.abs(xb).max(axis=2)
        if block == 32:
            bad = ~np.isfinite(xb).all(axis=2)
            _, e = np.frexp(np.where(bad, 1, b).astype(np.float64))
            k = np.where((b > 0) & ~bad, np.maximum(e - 3, -127), -127)
            v = e2m1(np.where(bad[:, :, None], 0, xb.astype(np.float64)) * np.exp2(-k)[:, :, None])
            v = v * np.where(bad, np.nan, np.exp2(k.astype(np.float64)))[:, :, None]
            g = np.ones(R)
        else:
            bad = ~np.isfinite(xb).all(axis=(1, 2))
            g = (np.where(bad, 0, b.max(axis=1)).astype(F) * F(1.0 / 2688.0)).astype(F)
            g = np.where(g < TINY, F(1), g)
            u = F(1) / g
            s = e4m3((b * u[:, None]).astype(F) * F(1.0 / 6.0))
            s = np.where(bad[:, None], 0.0, s)
            inv = np.where(s > 0, u[:, None] / np.where(s > 0, s, 1).astype(F), F(0)).astype(F)
            v = e2m1((np.where(bad[:, None, None], 0, xb) * inv[:, :, None]).astype(F)) * s[:, :, None]
            g = np.where(bad, np.nan, g.astype(np.float64))
    return v.reshape(R, -1)[:, :C], g


def fp4_values(x, block, bf16):
    """What reading back gives, bit for bit: (code * s) * g in float32, then the output type."""
    v, g = fp4(x, block)
    y = v.astype(F)
    if block == 16:
        y = y * g.astype(F)[:, None]
    return bf16_round(y) if bf16 else y


def fp4_matmul(a, b, block):
    """(exact float64 product, the sum of its terms' magnitudes) of float32 a [M,K], b [N,K]."""
    va, ga = fp4(a, block)
    vb, gb = fp4(b, block)
    return (va @ vb.T) * ga[:, None] * gb[None, :], (np.abs(va) @ np.abs(vb).T) * ga[:, None] * gb[None, :]
