"""The build's steps, on small sources: the library without PyTorch, the host module for the PyTorch at hand."""
import ctypes
import os
import sys

import pytest

from fp8_block_scaled_fp8bs_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    (src / "host.cpp").write_text("// nothing\n")
    monkeypatch.setattr(build, "CSRC", str(src))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libsmall.so"))
    monkeypatch.setattr(build, "HOST", str(tmp_path / "_host.so"))
    return tmp_path


def test_library_builds_without_pytorch(small, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)          # `import torch` fails
    lib = build.build()
    assert ctypes.CDLL(lib).one() == 1
    before = os.stat(lib).st_mtime_ns
    assert build.build() == lib and os.stat(lib).st_mtime_ns == before     # nothing to do, host module or not


def test_library_is_there_when_the_host_module_fails(small, monkeypatch):
    def fail():
        raise RuntimeError("no headers")
    monkeypatch.setattr(build, "build_host", fail)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build_all()
    assert ctypes.CDLL(build.LIB).one() == 1


def test_host_module_belongs_to_one_pytorch(small, monkeypatch):
    import torch
    host = small / "_host.so"
    assert not build.host_fits()
    host.write_bytes(b"")
    (small / "_host.so.txt").write_text(build._torch_tag())
    assert build.host_fits() and (os.utime(host) or build.host_up_to_date())
    monkeypatch.setattr(torch, "__version__", "1.0")
    assert not build.host_fits() and not build.host_up_to_date()
