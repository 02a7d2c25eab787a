"""What the build needs and what it rebuilds: the library without torch, the extension for the torch
that is there.  A stand-in for nvcc writes the outputs, so nothing is compiled."""
import os
import subprocess
import sys

import pytest

from continuous_batching_paged_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def here(tmp_path, monkeypatch):
    """The build in a folder of its own, with a compiler that touches what it is asked for."""
    for name in ("nvcc", "g++"):
        tool = tmp_path / "bin" / name
        tool.parent.mkdir(exist_ok=True)
        tool.write_text('#!/bin/sh\nwhile [ $# -gt 1 ]; do [ "$1" = -o ] && : > "$2"; shift; done\n')
        tool.chmod(0o755)
    monkeypatch.setenv("NVCC", str(tmp_path / "bin" / "nvcc"))
    monkeypatch.setenv("CXX", str(tmp_path / "bin" / "g++"))
    for name, path in (("BUILD_DIR", "_build"), ("LIB", "libcb.so"), ("EXT", "_cb_torch.so")):
        monkeypatch.setattr(_build, name, str(tmp_path / path))
    return tmp_path


def _hide_torch(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)


def test_both_are_built_once(here):
    assert _build.is_stale()
    assert _build.build() == str(here / "libcb.so")
    assert (here / "libcb.so").exists() and (here / "_cb_torch.so").exists()
    assert not _build.is_stale()


def test_library_builds_without_torch(here, monkeypatch):
    _hide_torch(monkeypatch)
    _build.build()
    assert (here / "libcb.so").exists() and not (here / "_cb_torch.so").exists()
    assert not _build.is_stale()


def test_library_is_linked_where_the_extension_does_not_compile(here, monkeypatch):
    monkeypatch.setenv("CXX", "/bin/false")         # (as without Python's or torch's headers)
    with pytest.raises(RuntimeError, match="cb_torch"):
        _build.build()
    assert (here / "libcb.so").exists()


def test_host_runtime_without_torch_and_extension():
    """Allocator and scheduler on the built library, torch hidden and the extension missing."""
    _build.build()
    code = """
import sys
sys.modules["torch"] = None
import continuous_batching_paged_gb300 as cb
from continuous_batching_paged_gb300 import _build
from continuous_batching_paged_gb300.runtime import BlockAllocator, Scheduler
_build.EXT += ".missing"
_build._compile = _build._compile_ext = None      # nothing has to be compiled
s = Scheduler(BlockAllocator(64, 16, 8), max_batch_tokens=64, max_requests_per_batch=4)
s.add_request(0, prompt_len=20, max_new_tokens=2)
assert int(s.step()["num_tokens"]) == 20
assert cb.workspace_size(1, 4, 2, 64, 20) > 0
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_extension_is_rebuilt_for_another_torch_or_python(here, monkeypatch):
    torch_dir = here / "torch"
    torch_dir.mkdir()
    (torch_dir / "version.py").write_text("__version__ = '1.0'\n")
    monkeypatch.setattr(_build, "_torch_dir", lambda: str(torch_dir))
    _build.build()
    assert not _build.is_stale()
    old = os.path.getmtime(torch_dir / "version.py")
    (torch_dir / "version.py").write_text("__version__ = '1.1'\n")
    os.utime(torch_dir / "version.py", (old - 1000, old - 1000))     # (files of packages keep their dates)
    assert _build.is_stale() and not _build.library_is_stale()
    _build.build()
    assert not _build.is_stale()
    monkeypatch.setattr(sys, "version", sys.version + " of another build")
    assert _build.is_stale() and not _build.library_is_stale()


def test_built_files_are_enough(here):
    # an installation that has the two libraries and not the build's folder compiles nothing
    _build.build()
    for f in (here / "_build").iterdir():
        f.unlink()
    (here / "_build").rmdir()
    assert not _build.is_stale()
