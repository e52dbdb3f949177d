"""Build libattn.so in-tree with nvcc for sm_103a (GB300).

Each .cu file compiles in parallel to an object under _build/, then the
shared libraries are linked next to this file:

* libattn.so -- the product: exports the functions of include/attn.h only
  (hidden visibility for everything else);
* libattn_test.so -- the same objects, with attn_api.cu compiled a second
  time with ATTN_TEST_EXPORTS, so that it also exports the test-only entry
  points of include/attn_test.h;
* libattn_checked.so -- the bounds-checking build: every source compiled
  with ATTN_BOUNDS_CHECK (and the test exports), so that the kernels test
  each global index and TMA coordinate before using it and report a failed
  test through the status word instead of touching memory out of bounds;
* _torch_calls.so -- the host side of the Python wrappers whose calls are
  short, against PyTorch's headers (csrc/torch_calls.cpp, by the host
  compiler).  Left out where either is missing: the wrappers then do without.

The CUDA runtime is linked statically (nvcc's default), so the libraries
need only the driver at run time; the tensor-map encoder is fetched from the
driver at first use.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libattn.so")
TEST_LIB = os.path.join(HERE, "libattn_test.so")
CHECKED_LIB = os.path.join(HERE, "libattn_checked.so")
CALLS_LIB = os.path.join(HERE, "_torch_calls.so")
SOURCES = ["attn_api.cu", "attn_bwd.cu", "attn_bwd_f32.cu", "attn_bwd_tc.cu", "attn_cache.cu", "attn_cache_fwd.cu", "attn_cache_select.cu",
           "attn_cache_tc.cu", "attn_f32.cu", "attn_rotary.cu", "attn_splitkv.cu", "attn_tc.cu"]
# (source, object name, extra flags) of the test library's own objects
TEST_SOURCES = [("attn_api.cu", "attn_api_test.o", ["-DATTN_TEST_EXPORTS"])]
# ... and of the bounds-checking library's, one per source
CHECKED_SOURCES = [(src, src.replace(".cu", "_checked.o"),
                    ["-DATTN_BOUNDS_CHECK"] + (["-DATTN_TEST_EXPORTS"] if src == "attn_api.cu"
                                               else []))
                   for src in SOURCES]
HEADERS = ["attn_bwd.h", "attn_internal.h", "cache_codec.cuh", "cache_fwd.cuh", "cache_index.h", "cache_mma.cuh",
           "sm100_ptx.cuh", "tc_common.cuh", "tensor_map.h"]
PUBLIC_HEADERS = ["attn.h", "attn_test.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return (ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-Xcompiler", "-fvisibility=hidden",
                    "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
            + list(extra))


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    deps = ([src] + [os.path.join(INCLUDE, h) for h in PUBLIC_HEADERS]
            + [os.path.join(CSRC, h) for h in HEADERS])
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir() -> str:
    """PyTorch's folder, found without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch not found")
    return list(spec.submodule_search_locations)[0]


def _torch_version():
    """Version of the PyTorch that is installed, or None."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


def _cxx():
    """The C++ compiler, or None."""
    return os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")


def _calls_compile(src: str, obj: str):
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    dirs = [INCLUDE, sysconfig.get_paths()["include"], inc,
            os.path.join(inc, "torch", "csrc", "api", "include"), cuda]
    return ([_cxx(), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w"]
            + [f for d in dirs for f in ("-I", d)] + ["-c", src, "-o", obj])


def _calls_link(lib: str, obj: str):
    # without libattn.so: it is handed the addresses of the one that is loaded
    return [_cxx(), "-shared", "-o", lib, obj, "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def _link(lib: str, objs) -> None:
    tmp = lib + ".tmp%d" % os.getpid()
    if lib == CALLS_LIB:
        cmd = _calls_link(tmp, *objs)
    else:
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + list(objs)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        print(r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, lib)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Builds the libraries (only what is stale); returns the product's path."""
    os.makedirs(BUILD, exist_ok=True)
    objs, jobs = {}, []
    units = ([(src, src.replace(".cu", ".o"), []) for src in SOURCES] + TEST_SOURCES
             + CHECKED_SOURCES)
    for src, oname, fl in units:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, oname)
        objs[oname] = o
        if force or _stale(o, s):
            jobs.append([nvcc()] + _flags(list(extra_flags) + fl) + ["-c", s, "-o", o])
    # one object for each version of PyTorch, whose headers it is made of
    version = _torch_version()
    calls_src = os.path.join(CSRC, "torch_calls.cpp")
    calls_obj = os.path.join(BUILD, "torch_calls-%s.o" % version)
    calls_job = None
    if version is None or _cxx() is None:
        print("%s is left out: %s not found" % (os.path.basename(CALLS_LIB),
                                                "PyTorch" if version is None else "a C++ compiler"))
    elif force or _stale(calls_obj, calls_src):
        calls_job = _calls_compile(calls_src, calls_obj)
    todo = jobs + ([calls_job] if calls_job else [])
    done = []
    if todo:
        with cf.ThreadPoolExecutor(max_workers=len(todo)) as ex:
            done = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), todo))

    def check(cmd, r):
        if verbose or r.returncode != 0:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("compiling %s failed" % cmd[-3])

    for cmd, r in zip(jobs, done):
        check(cmd, r)
    product = [objs[src.replace(".cu", ".o")] for src in SOURCES]
    test_set = product[:]
    for src, oname, _ in TEST_SOURCES:  # the test build replaces the product object
        test_set[SOURCES.index(src)] = objs[oname]
    if jobs or not os.path.exists(LIB) or force:
        _link(LIB, product)
    if jobs or not os.path.exists(TEST_LIB) or force:
        _link(TEST_LIB, test_set)
    if jobs or not os.path.exists(CHECKED_LIB) or force:
        _link(CHECKED_LIB, [objs[t[1]] for t in CHECKED_SOURCES])
    if calls_job:
        check(calls_job, done[-1])
    if version is not None and _cxx() is not None:
        stamp = os.path.join(BUILD, "torch_calls.version")  # of the PyTorch the library was linked for
        linked = open(stamp).read() if os.path.exists(stamp) else None
        if (calls_job or linked != version or not os.path.exists(CALLS_LIB)
                or os.path.getmtime(CALLS_LIB) < os.path.getmtime(calls_obj)):
            _link(CALLS_LIB, [calls_obj])
            with open(stamp, "w") as f:
                f.write(version)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ()))
