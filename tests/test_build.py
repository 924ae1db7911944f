"""What the build compiles and when, with compilers that only write their output file."""
import os
import subprocess
import types

import pytest

from paged_kv_cache_out_gb300 import build as cuda_build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A tree of empty sources; `ran` has the outputs made, `broken` the compilers that fail."""
    csrc, include, out = tmp_path / "csrc", tmp_path / "include", tmp_path / "_build"
    csrc.mkdir(), include.mkdir()
    for path in (csrc / "a.cu", csrc / "b.cu", csrc / "c.cuh", csrc / "torch_binding.cpp", include / "pkv.h"):
        path.write_text("")
        os.utime(path, (1, 1))
    for name, value in (("CSRC", csrc), ("INCLUDE", include), ("BUILD_DIR", out), ("LIB_PATH", out / "libpkv.so"),
                        ("EXT_SOURCE", csrc / "torch_binding.cpp"), ("EXT_PATH", out / "_pkv_torch.so")):
        monkeypatch.setattr(cuda_build, name, str(value))
    monkeypatch.setenv("CXX", "hostcxx")
    t = types.SimpleNamespace(path=tmp_path, ran=[], broken=())

    def run(cmd, **_):
        kind = "hostcxx" if cmd[0] == "hostcxx" else "nvcc"
        target = cmd[cmd.index("-o") + 1]
        if kind in t.broken:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="broken")
        with open(target, "w"):
            pass
        t.ran.append(os.path.basename(target).split(".tmp")[0])
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    return t


def exists(tree, name):
    return (tree.path / "_build" / name).exists()


def test_everything_once(tree):
    assert cuda_build.build() == cuda_build.LIB_PATH
    assert sorted(tree.ran) == ["_pkv_torch.so", "a.o", "b.o", "libpkv.so", "torch_binding.o"]
    assert tree.ran.index("libpkv.so") < tree.ran.index("_pkv_torch.so")
    tree.ran.clear()
    cuda_build.build()
    assert tree.ran == []


def test_the_library_does_not_wait_for_the_binding(tree):
    """A binding that does not compile is an error, but the library is there."""
    tree.broken = ("hostcxx",)
    with pytest.raises(RuntimeError, match="torch_binding.cpp"):
        cuda_build.build()
    assert exists(tree, "libpkv.so") and not exists(tree, "_pkv_torch.so")


def test_a_changed_binding_compiles_no_kernel(tree):
    cuda_build.build()
    tree.ran.clear()
    later = os.path.getmtime(cuda_build.EXT_PATH) + 10
    os.utime(cuda_build.EXT_SOURCE, (later, later))
    cuda_build.build()
    assert sorted(tree.ran) == ["_pkv_torch.so", "torch_binding.o"]


def test_a_changed_kernel_leaves_the_binding(tree):
    cuda_build.build()
    tree.ran.clear()
    later = os.path.getmtime(cuda_build.LIB_PATH) + 10
    os.utime(tree.path / "csrc" / "c.cuh", (later, later))
    cuda_build.build()
    assert sorted(tree.ran) == ["a.o", "b.o", "libpkv.so"]


def test_without_headers_there_is_a_library_and_a_warning(tree, monkeypatch):
    cuda_build.build()
    tree.ran.clear()
    later = os.path.getmtime(cuda_build.EXT_PATH) + 10
    os.utime(tree.path / "include" / "pkv.h", (later, later))
    monkeypatch.setattr(cuda_build.sysconfig, "get_paths", lambda: {"include": str(tree.path / "nowhere")})
    with pytest.warns(UserWarning, match="headers are missing"):
        assert cuda_build.build() == cuda_build.LIB_PATH
    assert sorted(tree.ran) == ["a.o", "b.o", "libpkv.so"]
    assert not exists(tree, "_pkv_torch.so")  # one of older sources would not fit


def test_a_failing_kernel_is_an_error(tree):
    tree.broken = ("nvcc",)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        cuda_build.build()
    assert not exists(tree, "libpkv.so")
