"""Refusals of the key-value cache's entry points, on the host, without a GPU."""
import ctypes

import pytest
import torch

P, ODD = ctypes.c_void_p(256), ctypes.c_void_p(260)
i64, vp, ci, cf, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class Cache(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("k", "v", "k_exp", "v_exp")] + [(n, i64) for n in ("pages", "kv_heads", "page",
                                                                                     "head_dim")]


class Batch(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("table", "lengths", "starts")] + [(n, i64) for n in ("batch", "width", "rows")]


CACHE = dict(k=256, v=256, k_exp=257, v_exp=259, pages=8, kv_heads=2, page=32, head_dim=64)
BATCH = dict(table=256, lengths=256, starts=256, batch=3, width=4, rows=5)
BAD_CACHE = [dict(k=None), dict(v=None), dict(k_exp=None), dict(v_exp=None), dict(k=264), dict(v=264), dict(pages=-1),
             dict(kv_heads=0), dict(kv_heads=-1), dict(kv_heads=2 ** 31), dict(pages=2 ** 31)]
ODD_CACHE = [dict(head_dim=96), dict(head_dim=256), dict(head_dim=0), dict(page=8), dict(page=24), dict(page=0)]
BAD_BATCH = [dict(table=None), dict(lengths=None), dict(starts=None), dict(batch=-1), dict(width=-1), dict(rows=-1),
             dict(width=2 ** 31 // 32), dict(rows=2 ** 30), dict(batch=2 ** 31), dict(batch=2 ** 29)]


@pytest.fixture(scope="module")
def qmm():
    import quantized_int8_matmul_gb300 as q
    lib = q.lib()
    lib.qmm_kv_append.argtypes = [vp, vp, ci, vp, i64, i64, vp, i64, i64, vp, i64, i64, i64, vp, vp, vp, i64, i64, ci, vp]
    lib.qmm_kv_read.argtypes = [vp, vp, vp, vp, ci, vp]
    lib.qmm_kv_attention.argtypes = [vp, vp, vp, ci, i64, i64, i64, cf, ci, i64, vp, vp, sz, vp]
    return q


def structs(cache, batch):
    return Cache(**{**CACHE, **cache}), Batch(**{**BATCH, **batch})


def append(q, cache=None, batch=None, dt=None, k=P, kr=128, kh=64, v=P, vr=128, vh=64, qp=P, qr=256, qh=64, heads=4,
           out=ctypes.c_void_p(512), cos=P, sin=P, pos=100, rot=32, inter=0):
    c, b = structs(cache or {}, batch or {})
    return q.lib().qmm_kv_append(ctypes.byref(c), ctypes.byref(b), q.QMM_F32 if dt is None else dt, k, kr, kh, v, vr, vh, qp,
                                 qr, qh, heads, out, cos, sin, pos, rot, inter, None)


def read(q, cache=None, batch=None, k=P, v=P, dt=None):
    c, b = structs(cache or {}, batch or {})
    return q.lib().qmm_kv_read(ctypes.byref(c), ctypes.byref(b), k, v, q.QMM_F32 if dt is None else dt, None)


def attention(q, cache=None, batch=None, qp=P, dt=None, qr=256, qh=64, heads=4, scale=0.1, causal=1, most=5,
              out=ctypes.c_void_p(512), ws=P, wb=2 ** 40):
    c, b = structs(cache or {}, batch or {})
    return q.lib().qmm_kv_attention(ctypes.byref(c), ctypes.byref(b), qp, q.QMM_F32 if dt is None else dt, qr, qh, heads,
                                    scale, causal, most, out, ws, wb, None)


@pytest.mark.parametrize("call", [append, read, attention])
def test_caches_and_batches(qmm, call):
    for kw in BAD_CACHE:
        assert call(qmm, cache=kw) == qmm.QMM_ERR_INVALID_ARG, kw
    for kw in ODD_CACHE:
        assert call(qmm, cache=kw) == qmm.QMM_ERR_UNSUPPORTED, kw
    for kw in BAD_BATCH:
        assert call(qmm, batch=kw) == qmm.QMM_ERR_INVALID_ARG, kw
    assert call(qmm, dt=qmm.QMM_S8) == qmm.QMM_ERR_INVALID_ARG
    for kw in (dict(rows=0), dict(batch=0)):
        assert call(qmm, batch=kw) == qmm.QMM_OK, kw
    empty = dict(rows=0, table=None, lengths=None)
    assert call(qmm, cache=dict(k=None, pages=0), batch=empty) == qmm.QMM_OK


def test_append_refusals(qmm):
    bad = qmm.QMM_ERR_INVALID_ARG
    for kw in (dict(k=None), dict(v=None), dict(out=None), dict(out=ODD), dict(cos=None), dict(sin=None), dict(cos=ODD),
               dict(sin=ODD), dict(kr=-1), dict(kh=-1), dict(vr=-1), dict(vh=-1), dict(qr=-1), dict(qh=-1), dict(heads=0),
               dict(heads=2 ** 30), dict(inter=2), dict(inter=-1), dict(rot=-16), dict(pos=-1), dict(pos=2 ** 31),
               dict(out=P, qr=257), dict(out=P, qh=65)):
        assert append(qmm, **kw) == bad, kw
    for rot in (80, 8, 24, 63):
        assert append(qmm, rot=rot) == qmm.QMM_ERR_UNSUPPORTED, rot
    lib = qmm.lib()
    c, b = structs({}, {})
    assert lib.qmm_kv_read(None, ctypes.byref(b), P, P, qmm.QMM_F32, None) == bad
    assert lib.qmm_kv_read(ctypes.byref(c), None, P, P, qmm.QMM_F32, None) == bad


def test_read_refusals(qmm):
    for kw in (dict(k=ODD), dict(v=ODD)):
        assert read(qmm, **kw) == qmm.QMM_ERR_INVALID_ARG, kw
    assert read(qmm, k=None, v=None) == qmm.QMM_OK


def test_attention_refusals(qmm):
    bad = qmm.QMM_ERR_INVALID_ARG
    for kw in (dict(qp=None), dict(out=None), dict(out=ODD), dict(out=P), dict(qr=-1), dict(qh=-1), dict(heads=0), dict(heads=3),
               dict(heads=2 ** 30), dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2), dict(most=0),
               dict(ws=None), dict(ws=ODD)):
        assert attention(qmm, **kw) == bad, kw
    ws = qmm.lib().qmm_kv_attention_workspace_bytes
    for args in ((-1, 1, 4, 2, 64, 0, 1), (1, -1, 4, 2, 64, 0, 1), (1, 1, 3, 2, 64, 0, 1), (1, 1, 4, 0, 64, 0, 1),
                 (1, 1, 4, 2, 65, 0, 1), (1, 1, 4, 2, 64, 2, 1), (1, 1, 4, 2, 64, 0, 0), (0, 1, 4, 2, 64, 0, 1),
                 (1, 0, 4, 2, 64, 0, 1)):
        assert ws(*args) == 0, args


def test_python_refusals(qmm):
    """What the binding refuses before any pointer is taken (CPU tensors stand in)."""
    with pytest.raises(ValueError, match="head_dim"):
        qmm.qmm_kv_cache(4, 2, 80)
    with pytest.raises(ValueError, match="page"):
        qmm.qmm_kv_cache(4, 2, 64, page=40)
    c = qmm.qmm_kv_cache(4, 2, 64, page=32, device="cpu")
    assert c.k.shape == (4, 2, 32, 64) and c.k_exp.shape == (4, 2, 2)
    x, t, n = torch.zeros(3, 2, 64), torch.zeros(3, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        qmm.qmm_kv_append(c, x, x, t, n)
    with pytest.raises(ValueError, match="CUDA"):
        qmm.qmm_kv_read(c, t, n)
    with pytest.raises(ValueError, match="CUDA"):
        qmm.qmm_kv_attention(x, c, t, n)
    with pytest.raises(ValueError, match="rows"):
        qmm.qmm_kv_read(c, t, n, starts=n)
