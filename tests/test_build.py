"""The library and the compiled binding are built apart: the layer needs none of the binding's tools."""
import os
import subprocess
import sys

import pytest
import torch

from memory_bound_cnn_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def child(code, **env):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, env={**os.environ, **env}, capture_output=True, text=True)


@pytest.mark.parametrize("cxx", ["false", "no-such-compiler"])  # one that fails, and none
def test_the_layer_loads_without_the_binding(tmp_path, cxx):
    """The library is there, the binding is not and cannot be built: the layer loads, and only what needs
    the binding raises."""
    _build.build()
    code = f"""
from memory_bound_cnn_gb300 import _build, wtconv
_build.BINDING = {str(tmp_path / "_binding.so")!r}
print(wtconv.wtconv_version() >= 0)
try:
    wtconv.load_binding()
except RuntimeError as e:
    print("refused")
"""
    r = child(code, CXX=cxx)
    assert r.returncode == 0 and r.stdout.split() == ["True", "refused"], r.stdout + r.stderr


def test_the_library_is_linked_where_the_binding_fails(tmp_path):
    _build.build()
    code = f"""
import os
from memory_bound_cnn_gb300 import _build
_build.BINDING, _build.LIB = {str(tmp_path / "_binding.so")!r}, {str(tmp_path / "libwtconv.so")!r}
try:
    _build.build()
except RuntimeError:
    print("refused", os.path.exists(_build.LIB))
"""
    r = child(code, CXX="false")
    assert r.returncode == 0 and r.stdout.split() == ["refused", "True"], r.stdout + r.stderr


def test_another_pytorch_makes_the_binding_stale(monkeypatch):
    """The binding holds PyTorch's and Python's layouts: it is rebuilt when either changes, not reused."""
    _build.build()
    assert not _build.binding_stale()
    for module, name, value in ((torch, "__version__", "1.0"), (torch._C, "_GLIBCXX_USE_CXX11_ABI", None)):
        with monkeypatch.context() as m:
            m.setattr(module, name, value)
            assert _build.binding_stale(), name
    assert not _build.binding_stale()
