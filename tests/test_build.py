"""The build without torch, and the Python binding without its C++ path."""
import importlib.util
import os
import sys

import pytest
import torch

import int4_dequantize_matmul_amd as q4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build.py by its path, with empty output folders and commands that only write their output file."""
    spec = importlib.util.spec_from_file_location("build_alone", os.path.join(ROOT, "int4_dequantize_matmul_amd", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for name in ("BUILD", "LIBDIR", "LIB", "TORCH_LIB", "PROBE_LIB"):
        monkeypatch.setattr(m, name, str(tmp_path / os.path.basename(getattr(m, name))))
    for name in ("LIB", "TORCH_LIB", "PROBE_LIB"):
        monkeypatch.setattr(m, name, os.path.join(m.LIBDIR, os.path.basename(getattr(m, name))))
    m.fail = ""

    def run(cmd):
        out = cmd[cmd.index("-o") + 1]
        if m.fail and m.fail in out:
            raise RuntimeError("build step failed")
        open(out, "w").close()
        return ""
    monkeypatch.setattr(m, "_run", run)
    return m


def test_the_library_is_built_without_torch(build, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)      # import torch raises
    assert build.build() == build.LIB
    assert sorted(os.listdir(build.LIBDIR)) == ["libq4.so", "libq4_probe.so"]


def test_the_binding_is_built_with_torch(build):
    build.build()
    assert sorted(os.listdir(build.LIBDIR)) == ["libq4.so", "libq4_probe.so", "q4_torch.so"]


def test_a_binding_that_does_not_compile_is_an_error_and_leaves_the_library(build):
    build.fail = "q4_torch"
    with pytest.raises(RuntimeError):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.TORCH_LIB)


@pytest.fixture
def unbound(monkeypatch):
    monkeypatch.setattr(q4, "_DIRECT", None)


def check_ctypes_path():
    with pytest.warns(RuntimeWarning, match="ctypes"):
        with pytest.raises(TypeError):      # the ctypes path's own checks
            q4.q4_mx_quantize_rows(torch.zeros(2, 32))
    with pytest.raises(TypeError):          # said once
        q4.q4_linear_w4a16_mx(torch.zeros(2, 32), None, None)


def test_a_missing_binding_leaves_the_ctypes_path(unbound, monkeypatch, tmp_path):
    monkeypatch.setattr(q4, "TORCH_LIB_PATH", str(tmp_path / "q4_torch.so"))
    check_ctypes_path()


def test_a_binding_that_does_not_load_leaves_the_ctypes_path(unbound, monkeypatch, tmp_path):
    (tmp_path / "q4_torch.so").write_bytes(b"not a library")
    monkeypatch.setattr(q4, "TORCH_LIB_PATH", str(tmp_path / "q4_torch.so"))
    check_ctypes_path()


def test_a_binding_for_another_torch_leaves_the_ctypes_path(unbound, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    check_ctypes_path()


def test_the_binding_in_the_tree_is_bound(unbound, recwarn):
    assert q4._direct().built_for.startswith("torch ")
    assert not [w for w in recwarn if "ctypes" in str(w.message)]
