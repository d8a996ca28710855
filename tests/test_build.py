"""The build step on the CPU, with a stand-in for the compiler."""

import os
import stat
import subprocess

import pytest

from paged_kv_cache_210_gb300 import build as lib_build


@pytest.fixture
def compiler(tmp_path, monkeypatch):
    """A compiler that writes its output and fails for one source (or for the link); the
    build's folder is an empty one."""
    def make(fails):
        script = tmp_path / "nvcc"
        script.write_text('#!/bin/sh\nout=""\nfor a in "$@"; do [ "$last" = -o ] && out="$a"; last="$a"; '
                          'done\necho made > "$out"\ncase "$*" in ' + fails + ') exit 1;; esac\n')
        script.chmod(script.stat().st_mode | stat.S_IXUSR)
        monkeypatch.setattr(lib_build, "nvcc", lambda: str(script))
        folder = tmp_path / "_build"
        monkeypatch.setattr(lib_build, "BUILD_DIR", str(folder))
        monkeypatch.setattr(lib_build, "LIBRARY", str(folder / "libpkv.so"))
        return folder
    return make


@pytest.mark.parametrize("fails", ["*csrc/tree.cu*", "*csrc/axes.cu*", "*-shared*"])
def test_a_failed_build_leaves_nothing(compiler, fails):
    folder = compiler(fails)
    with pytest.raises(subprocess.CalledProcessError):
        lib_build.build()
    assert os.listdir(folder) == []


def test_a_build_leaves_the_library_alone(compiler):
    folder = compiler("nothing")
    assert lib_build.build() == str(folder / "libpkv.so")
    assert os.listdir(folder) == ["libpkv.so"]
    before = os.stat(folder / "libpkv.so").st_mtime_ns
    lib_build.build()                              # not stale
    assert os.stat(folder / "libpkv.so").st_mtime_ns == before
