"""The native module belongs to one Python and one torch: it is built again for another,
and where it cannot be built or loaded the package loads without it and only the calls
that need it fail."""
import os
import subprocess
import sys

import pytest

import quantized_int8_matmul_gb300 as q
from quantized_int8_matmul_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_another_torch_or_python_makes_it_stale(monkeypatch):
    assert not _build.needs_build()
    tag = _build.binding_tag()
    import torch
    assert torch.__version__ in tag
    monkeypatch.setattr(_build, "binding_tag", lambda: tag + "x")
    assert _build.binding_stale() and _build.needs_build() and not _build.library_stale()


def test_a_torch_without_cuda_is_refused_before_compiling(monkeypatch, tmp_path):
    (tmp_path / "lib").mkdir()
    (tmp_path / "version.py").write_text("__version__ = 'none'\n")
    monkeypatch.setattr(_build, "_torch_dir", lambda: str(tmp_path))
    monkeypatch.setattr(_build, "_compile", lambda src: pytest.fail("compiled"))
    with pytest.raises(RuntimeError, match="CUDA"):
        _build.build_binding()


def test_the_package_loads_without_it():
    code = """
import sys
sys.modules["quantized_int8_matmul_gb300._binding"] = None      # importing it fails
import torch
import quantized_int8_matmul_gb300 as q
print(q.qmm_a8w8_workspace_bytes(4096, 4096, 4096) > 0, q.qmm_fp4_bytes(128, 128, 16))
try:
    q.qmm_a8w8(torch.zeros(2, 2), torch.zeros(2, 2), torch.zeros(2), torch.zeros(2))
except ValueError as e:
    print(e)
for f in (lambda: q.qmm_rms_norm_s8(torch.zeros(2, 8), torch.zeros(8)), lambda: q.qmm_fp4_quantize(torch.zeros(2, 8))):
    try:
        f()
    except RuntimeError as e:
        print(type(e).__name__, "_binding" in str(e))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.splitlines() == [f"True {q.qmm_fp4_bytes(128, 128, 16)}", "A must be a CUDA tensor",
                                     "RuntimeError True", "RuntimeError True"]


def test_the_module_goes_without_the_build_folder(monkeypatch, tmp_path):
    """A tree shipped with its two libraries and not the objects is not stale."""
    assert os.path.dirname(_build.BINDING_TAG) == os.path.dirname(_build.BINDING_PATH)
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path / "none"))
    assert not _build.needs_build()
