"""The bulk copies of rows off 16 bytes stay inside their tensor: the extents that the
kernels use (a header without device code), compiled for the host and walked over every
row of tensors of every width and type."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def row_copy_bytes(tmp_path_factory):
    d = tmp_path_factory.mktemp("row_copy")
    src = d / "f.cpp"
    src.write_text('#include "row_copy.h"\nextern "C" unsigned f(int n, int s, int size, int last) {\n'
                   "  return qmm::row_copy_bytes(n, s, size, last != 0);\n}\n")
    inc = os.path.join(ROOT, "quantized_int8_matmul_gb300", "csrc")
    subprocess.run([os.environ.get("CXX", "g++"), "-shared", "-fPIC", "-I" + inc, str(src), "-o", str(d / "f.so")],
                   check=True)
    f = ctypes.CDLL(str(d / "f.so")).f
    f.restype = ctypes.c_uint
    return f


@pytest.mark.parametrize("size", [2, 4])
@pytest.mark.parametrize("gap", [0, 1, 3])    # 16-byte units between rows
def test_copies_stay_inside_the_tensor(row_copy_bytes, size, gap):
    E = 16 // size
    for n in list(range(32 * E + 1, 32 * E + 2 * E + 1)) + [4095, 4096, 4099, 5003, 12285]:
        for M in (1, 2, 3, 8, 11):
            ld = n + gap * E
            extent = ((M - 1) * ld + n) * size        # bytes of the caller's tensor
            for m in range(M):
                s = (m * n) % E                        # the row's start past a 16-byte boundary
                assert (m * ld - s) * size % 16 == 0
                first = (m * ld - s) * size
                count = row_copy_bytes(n, s, size, m == M - 1)
                assert first >= 0 and count % 16 == 0 and first + count <= extent
                left = (m * ld + n) * size - (first + count)
                assert left < 16 and (left <= 0 or m == M - 1)   # the row, but for the last one's end
