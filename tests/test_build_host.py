"""The build: libattn.so needs nvcc and nothing else; the wrappers' host side is built where PyTorch and a
C++ compiler are there, and the wrappers do without it where they are not."""
import importlib.metadata
import os

import pytest
import torch

import online_softmax_forward_gb300 as pkg
from online_softmax_forward_gb300 import build as lib_build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """Libraries are linked in a folder of their own, from the objects that are there."""
    lib_build.build()
    for name in ("LIB", "TEST_LIB", "CHECKED_LIB", "CALLS_LIB"):
        monkeypatch.setattr(lib_build, name, str(tmp_path / os.path.basename(getattr(lib_build, name))))
    return tmp_path


def without_torch(monkeypatch):
    def version(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", version)


def without_compiler(monkeypatch):
    which = lib_build.shutil.which
    monkeypatch.setattr(lib_build.shutil, "which", lambda name, **kw: which(name, **kw) if name == "nvcc" else None)
    monkeypatch.delenv("CXX", raising=False)


@pytest.mark.parametrize("missing", [without_torch, without_compiler])
def test_cuda_libraries_need_nvcc_alone(elsewhere, monkeypatch, missing):
    missing(monkeypatch)
    assert lib_build.build() == str(elsewhere / "libattn.so")
    assert sorted(os.listdir(elsewhere)) == ["libattn.so", "libattn_checked.so", "libattn_test.so"]


def test_a_failed_compilation_of_the_host_side_comes_after_the_libraries(elsewhere, monkeypatch):
    monkeypatch.setattr(lib_build, "_calls_compile", lambda src, obj: ["false", "-c", src, "-o", obj])
    monkeypatch.setattr(lib_build, "_stale", lambda obj, src: src.endswith(".cpp"))
    with pytest.raises(RuntimeError, match="torch_calls.cpp"):
        lib_build.build()
    assert (elsewhere / "libattn.so").exists()


def test_wrappers_do_without_the_host_side(monkeypatch, tmp_path):
    monkeypatch.setattr(pkg, "_calls", None)
    monkeypatch.setattr(pkg, "_HERE", str(tmp_path))
    with pytest.warns(RuntimeWarning, match="_torch_calls.so"):
        calls = pkg._fast()
    q, pos = torch.zeros(1, 2, 3, 64), torch.zeros(1, 3, dtype=torch.int32)
    assert calls.rotary(q, None, pos, False) is None and calls.attention_bwd(q, q, q, q, q, q, None, False, 0.0) is None
    with pytest.raises(ValueError, match="CUDA"):
        pkg.attention_bwd(q, q, q, q, torch.zeros(1, 2, 3), q)


def test_the_host_side_follows_the_version_of_torch(elsewhere, monkeypatch):
    """Built for one PyTorch, then for another, then for the first again: each time that one's object."""
    links = []
    monkeypatch.setattr(lib_build, "_link", lambda lib, objs: (links.append(list(objs)), open(lib, "w").close()))
    objects = {v: os.path.join(lib_build.BUILD, "torch_calls-%s.o" % v) for v in ("0.0.1", "0.0.2")}
    monkeypatch.setattr(lib_build, "_stale", lambda obj, src: src.endswith(".cpp") and not os.path.exists(obj))
    monkeypatch.setattr(lib_build, "_calls_compile", lambda src, obj: ["cp", src, obj])
    try:
        for v in ("0.0.1", "0.0.2", "0.0.1", "0.0.1"):
            monkeypatch.setattr(lib_build, "_torch_version", lambda v=v: v)
            lib_build.build()
        calls = [objs[0] for objs in links if "torch_calls" in objs[0]]
        assert calls == [objects["0.0.1"], objects["0.0.2"], objects["0.0.1"]]
    finally:
        for path in objects.values():
            if os.path.exists(path):
                os.remove(path)
