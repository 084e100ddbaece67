"""Pointers of the key-value cache's calls that do not lie on their elements are refused, on the host."""
import ctypes

import pytest

from test_kv_abi import append, attention, qmm, read  # noqa: F401

OFF = [ctypes.c_void_p(256 + n) for n in (1, 2, 3)]


@pytest.mark.parametrize("call", [append, read, attention])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_integers(qmm, call, off):  # noqa: F811
    for kw in (dict(table=256 + off), dict(lengths=256 + off), dict(starts=256 + off)):
        assert call(qmm, batch=kw) == qmm.QMM_ERR_INVALID_ARG, kw


def test_rows(qmm):  # noqa: F811
    for p in OFF:
        for kw in (dict(k=p), dict(v=p), dict(qp=p)):
            assert append(qmm, **kw) == qmm.QMM_ERR_INVALID_ARG, (kw, p)
            if p.value % 2:
                assert append(qmm, dt=qmm.QMM_BF16, **kw) == qmm.QMM_ERR_INVALID_ARG, (kw, p)
        assert attention(qmm, qp=p) == qmm.QMM_ERR_INVALID_ARG
        if p.value % 2:
            assert attention(qmm, qp=p, dt=qmm.QMM_BF16) == qmm.QMM_ERR_INVALID_ARG
