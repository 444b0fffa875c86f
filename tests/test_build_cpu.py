"""The C library and the package without the binding's C++ part, and the C++ part of
another PyTorch: no compiler runs here."""

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "nvfp4_weight_quantized_moe_b200"


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    mod = __graft_entry__._build_module()
    mod.build()
    return mod


@pytest.fixture
def bare(built, tmp_path):
    """The package with its library and without a C++ part."""
    shutil.copytree(os.path.join(ROOT, PKG), tmp_path / PKG, ignore=shutil.ignore_patterns("_quick_call*", "__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    os.utime(tmp_path / PKG / "libnvfp4moe.so")  # newer than the copied sources
    return tmp_path


def _python(cwd, code):
    return subprocess.run([sys.executable, "-c", code], cwd=cwd, capture_output=True, text=True, timeout=300)


IMPORT = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import nvfp4_weight_quantized_moe_b200._binding as B
print(len([w for w in seen if "C++ part" in str(w.message)]), B._quick_call is None)
import torch
try:
    B.route_topk(torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
except ValueError as e:
    print(e)
"""


def test_the_package_imports_without_the_extension(bare):
    res = _python(bare, IMPORT)
    assert res.returncode == 0, res.stderr[-2000:]
    assert res.stdout.splitlines() == ["1 True", "logits: must be a CUDA tensor"]


def test_another_pytorch_s_extension_is_not_loaded(bare, built):
    """Built against another version, it may load and read tensors wrongly."""
    name = os.path.basename(built.quick_call_path("0.0.1"))
    (bare / PKG / name).write_bytes(b"not this one")
    res = _python(bare, IMPORT)
    assert res.returncode == 0 and res.stdout.startswith("1 True"), res.stderr[-2000:]
    assert built.quick_call_path("2.0.0") != built.quick_call_path("2.0.1")


def test_an_extension_that_does_not_load_is_said_and_left(bare, built):
    import torch
    name = os.path.basename(built.quick_call_path(torch.__version__))
    (bare / PKG / name).write_bytes(b"no shared object")
    res = _python(bare, IMPORT)
    assert res.returncode == 0 and res.stdout.startswith("1 True"), res.stderr[-2000:]


def test_the_library_builds_where_there_is_no_pytorch(bare):
    code = f"""
import importlib.util, sys
sys.modules["torch"] = None          # every import of it fails
spec = importlib.util.spec_from_file_location("b", {str(bare / PKG / "build.py")!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
print(b.build() == b.LIB_PATH)
"""
    res = _python(bare, code)
    assert res.returncode == 0 and res.stdout == "True\n", res.stderr[-2000:]
    assert "C++ part is not built" in res.stderr


def test_the_tree_s_own_extension_is_loaded(built):
    import nvfp4_weight_quantized_moe_b200._binding as B
    assert B._quick_call is not None
