"""The in-tree build, on a library of one small file in a folder of its own: the library does not hang on its binding.
The binding's name, which says what it was built against."""
import ctypes
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn
from gated_deltanet_linear_gdn_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """build.py's places moved to tmp_path, with one source."""
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    for name, value in dict(CSRC=str(src), BUILD_DIR=str(tmp_path / "o"), LIB=str(tmp_path / "libsmall.so"),
                            binding_path=lambda: str(tmp_path / "_binding.so"), SOURCES=["one.cu"]).items():
        monkeypatch.setattr(build, name, value)
    return tmp_path


def command(out):
    return ["cp", os.path.abspath(__file__), out]


def test_a_binding_that_does_not_compile(small, monkeypatch):
    for why in (lambda out: ["sh", "-c", "echo no such header; exit 1"], lambda out: ["/nonexistent/g++", out]):
        monkeypatch.setattr(build, "_binding_command", why)
        with pytest.raises(RuntimeError, match="is built, its binding for Python failed"):
            build.build_library(force=True)
        assert ctypes.CDLL(build.LIB).one() == 1
        os.remove(build.LIB)
    assert not os.path.exists(build.binding_path())


def test_a_library_without_its_binding(small, monkeypatch):
    monkeypatch.setattr(build, "_binding_command", None)        # (not called)
    assert build.stale(binding=False)
    assert build.build_library(binding=False) == build.LIB
    assert not build.stale(binding=False) and build.stale()
    assert ctypes.CDLL(build.LIB).one() == 1


def test_a_library_that_does_not_compile(small, monkeypatch):
    monkeypatch.setattr(build, "_binding_command", command)
    (small / "csrc" / "one.cu").write_text("no code\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build_library()
    assert not os.path.exists(build.LIB) and not [f for f in os.listdir(small) if ".tmp" in f]


def test_both_and_again(small, monkeypatch):
    monkeypatch.setattr(build, "_binding_command", command)
    assert build.stale()
    build.build_library()
    assert not build.stale() and os.path.exists(build.binding_path())
    assert not [f for f in os.listdir(small) if ".tmp" in f]
    then = os.path.getmtime(build.LIB)
    build.build_library()
    assert os.path.getmtime(build.LIB) == then
    os.utime(small / "csrc" / "one.cu", (then + 5, then + 5))
    assert build.stale()


def test_the_binding_is_of_one_torch_and_one_python(monkeypatch):
    """Under another version the binding that is there is not taken: building makes one, and without that the first call says
    that it is missing instead of failing in its symbols."""
    build.build_library()
    assert not build.stale() and gdn.BINDING_PATH == build.binding_path() and os.path.exists(build.binding_path())
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "99.0")
        assert build.stale() and not build.stale(binding=False)
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-999")
        assert build.stale()
    code = """import torch; torch.__version__ = "99.0"
import gated_deltanet_linear_gdn_gb300 as gdn
x = torch.zeros(1, 1, 2, dtype=torch.bfloat16)
try: gdn.gdn_rope(x, None, x, x, None, gdn.RopeTable(2, device="cpu"))
except RuntimeError as e: assert "for this torch and this Python" in str(e), e
else: raise SystemExit(1)"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=build.ROOT)
