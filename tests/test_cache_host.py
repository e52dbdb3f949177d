"""The paged 8-bit cache on the host: the index arithmetic its kernels share
(csrc/cache_index.h, compiled here with the C++ compiler), refusals of every
entry point before any CUDA call, and the Python wrappers' checks."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import online_softmax_forward_gb300 as pkg
from online_softmax_forward_gb300 import build as lib_build

SHIM = """
#include "cache_index.h"
using namespace attn;
extern "C" {
int64_t begin_(int64_t w, int64_t t, int64_t n) { return worker_begin(w, t, n); }
int64_t of_(int64_t x, int64_t t, int64_t n) { return worker_of(x, t, n); }
int64_t count_(int64_t t, int64_t most, int64_t least) { return worker_count(t, most, least); }
int clamp_(int len, int pages, int page) { return clamp_len(len, pages, page); }
int visible_(int len, int cnt, int i, int causal) { return visible_keys(len, cnt, i, causal); }
uint32_t div_(uint32_t n, uint32_t d) { return n / fast_div(d); }
void advance_(int *p, int by, int units, const int *tiles) {
    Place q = {p[0], p[1], p[2], p[3]};
    advance(q, by, units, [&](int b) { return tiles[b]; });
    p[0] = q.b; p[1] = q.unit; p[2] = q.t; p[3] = q.n;
}
int64_t touched_(int64_t s, int page) { return touched_pages(s, page); }
}
"""


@pytest.fixture(scope="module")
def idx(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx, "a C++ compiler is part of the build"
    d = tmp_path_factory.mktemp("cache_index")
    src, so = str(d / "shim.cpp"), str(d / "shim.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", lib_build.CSRC, src, "-o", so],
                   check=True)
    lib = ctypes.CDLL(so)
    for name, res, args in (("begin_", 8, (8, 8, 8)), ("of_", 8, (8, 8, 8)), ("count_", 8, (8, 8, 8)),
                            ("clamp_", 4, (4, 4, 4)), ("visible_", 4, (4, 4, 4, 4)),
                            ("touched_", 8, (8, 4))):
        t = {8: ctypes.c_int64, 4: ctypes.c_int}
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = t[res], [t[a] for a in args]
    lib.div_.restype, lib.div_.argtypes = ctypes.c_uint32, [ctypes.c_uint32] * 2
    ints = ctypes.POINTER(ctypes.c_int)
    lib.advance_.restype, lib.advance_.argtypes = None, [ints, ctypes.c_int, ctypes.c_int, ints]
    return lib


def test_division_by_multiplication(idx):
    top = 2 ** 31 - 1
    for d in (1, 2, 3, 5, 7, 8, 9, 127, 128, 129, 1000, 65535, 65536, 99991, 2 ** 30, 2 ** 30 + 1, top):
        for k in (0, 1, 2, 3, top // d // 2, top // d):
            for n in (k * d - 1, k * d, k * d + 1, k * d + d - 1, top):
                if 0 <= n <= top:
                    assert idx.div_(n, d) == n // d, (n, d)


@pytest.mark.parametrize("tiles", [[3], [1, 0, 2], [0, 5, 0, 0, 1, 7], [1] * 9])
@pytest.mark.parametrize("units", [1, 2, 5])
@pytest.mark.parametrize("by", [1, 4, 32])
def test_advance_steps_through_the_units(idx, tiles, units, by):
    order = [(b, u, t, n) for b, n in enumerate(tiles) for u in range(units) for t in range(n)]
    c = (ctypes.c_int * len(tiles))(*tiles)
    for start in range(len(order)):
        if start + by < len(order):
            p = (ctypes.c_int * 4)(*order[start])
            idx.advance_(p, by, units, c)
            assert tuple(p) == order[start + by]


@pytest.mark.parametrize("workers", [1, 2, 7, 1216, 1280])
@pytest.mark.parametrize("total", [1, 2, 5, 1215, 1216, 1217, 5000, 99991])
def test_worker_ranges_cover_every_tile_once(idx, total, workers):
    n = idx.count_(total, workers, 1)
    assert 1 <= n <= workers and n <= total
    edges = [idx.begin_(w, total, n) for w in range(n + 1)]
    assert edges[0] == 0 and edges[-1] == total
    sizes = [b - a for a, b in zip(edges, edges[1:])]
    assert min(sizes) >= 1 and max(sizes) - min(sizes) <= 1
    w = 0
    for x in range(total):
        while x >= edges[w + 1]:
            w += 1
        assert idx.of_(x, total, n) == w


def test_worker_arithmetic_at_the_largest_totals(idx):
    total, n = 2 ** 51 - 3, 1280
    edges = [idx.begin_(w, total, n) for w in range(n + 1)]
    assert edges[0] == 0 and edges[-1] == total and edges == sorted(edges)
    for w in (0, 1, 639, 1279):
        assert idx.of_(edges[w], total, n) == w
        assert idx.of_(edges[w + 1] - 1, total, n) == w


def test_worker_count_keeps_the_least_range(idx):
    assert idx.count_(0, 1216, 1) == 1
    assert idx.count_(10, 1216, 4) == 3
    assert idx.count_(10 ** 6, 1216, 4) == 1216


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_touched_pages_is_the_largest_number(idx, page):
    for S in (1, 2, page - 1, page, page + 1, 2 * page, 3 * page + 5):
        most = max((pos + S - 1) // page - pos // page + 1 for pos in range(page))
        assert idx.touched_(S, page) == most
    assert idx.touched_(0, page) == 0


def test_lengths_are_clamped_to_the_table(idx):
    assert idx.clamp_(-5, 4, 16) == 0
    assert idx.clamp_(64, 4, 16) == 64
    assert idx.clamp_(65, 4, 16) == 64
    assert idx.clamp_(2 ** 31 - 1, 2 ** 31 - 1, 128) == 2 ** 31 - 1  # the capacity passes 2^31


def test_visible_keys(idx):
    # len, cnt, i, causal
    assert [idx.visible_(10, 3, i, 1) for i in range(4)] == [8, 9, 10, 0]
    assert [idx.visible_(10, 3, i, 0) for i in range(4)] == [10, 10, 10, 0]
    assert idx.visible_(2, 5, 0, 1) == 0 and idx.visible_(2, 5, 4, 1) == 2  # rows before the first token
    assert idx.visible_(0, 1, 0, 1) == 0 and idx.visible_(0, 1, 0, 0) == 0


# ------------------------------------------------------------------ refusals
K, V, KS, VS, KB = 0x1000000, 0x2000000, 0x3000000, 0x3100000, 0x3200000
NK, NV, Q, O, L = 0x4000000, 0x5000000, 0x6000000, 0x7000000, 0x8000000
TABLE, LENS, COUNTS, PAGES, WS = 0x9000000, 0x9100000, 0x9200000, 0x9300000, 0xA000000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return pkg.load_library()


def cache(**kw):
    c = dict(k=K, v=V, k_scale=KS, v_scale=VS, k_bounds=KB, n_pages=8, H_kv=2, page=16, d=64, format=0)
    c.update(kw)
    return pkg._Cache(*(c[f] for f, _ in pkg._Cache._fields_))


def append(lib, c=None, **kw):
    a = dict(k=NK, v=NV, table=TABLE, max_pages=4, pos=LENS, counts=COUNTS, B=2, S=3, dtype=pkg.ATTN_BF16)
    a.update(kw)
    return lib.attn_cache_append(cache() if c is None else c, a["k"], a["v"], a["table"], a["max_pages"],
                                 a["pos"], a["counts"], a["B"], a["S"], a["dtype"], None)


def read(lib, c=None, **kw):
    a = dict(table=TABLE, max_pages=4, lens=LENS, k=NK, v=NV, B=2, S=30, dtype=pkg.ATTN_F16)
    a.update(kw)
    return lib.attn_cache_read(cache() if c is None else c, a["table"], a["max_pages"], a["lens"], a["k"],
                               a["v"], a["B"], a["S"], a["dtype"], None)


def select(lib, c=None, **kw):
    a = dict(q=Q, table=TABLE, max_pages=4, lens=LENS, counts=None, pages=PAGES, n=2, B=2, H=4, Sq=1,
             causal=1, dtype=pkg.ATTN_BF16, ws=WS, bytes=1 << 20)
    a.update(kw)
    return lib.attn_cache_select(cache() if c is None else c, a["q"], a["table"], a["max_pages"], a["lens"],
                                 a["counts"], a["pages"], a["n"], a["B"], a["H"], a["Sq"], a["causal"],
                                 a["dtype"], a["ws"], a["bytes"], None)


def attend(lib, c=None, **kw):
    a = dict(q=Q, o=O, lse=L, table=TABLE, max_pages=4, lens=LENS, counts=COUNTS, pages=None, n=0, B=2, H=4,
             Sq=1, causal=1, scale=0.0, dtype=pkg.ATTN_BF16, ws=WS, bytes=BIG)
    a.update(kw)
    return lib.attn_fwd_cache(cache() if c is None else c, a["q"], a["o"], a["lse"], a["table"],
                              a["max_pages"], a["lens"], a["counts"], a["pages"], a["n"], a["B"], a["H"],
                              a["Sq"], a["causal"], a["scale"], a["dtype"], a["ws"], a["bytes"], None)


CALLS = {"append": append, "read": read, "select": select, "attend": attend}


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
@pytest.mark.parametrize("name", CALLS)
def test_valid_arguments_reach_the_device_check(lib, name):
    assert CALLS[name](lib) == pkg.ATTN_ERR_UNSUPPORTED_DEVICE


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(k=K + 8), dict(v=V + 1),
    dict(k_scale=KS + 2), dict(k_bounds=KB + 4), dict(n_pages=0), dict(n_pages=-1), dict(H_kv=0),
    dict(page=8), dict(page=48), dict(page=256), dict(d=32), dict(d=96), dict(d=256), dict(format=2),
    dict(format=-1), dict(n_pages=1 << 30, H_kv=4),
], ids=lambda kw: ",".join("%s=%s" % i for i in kw.items()))
def test_bad_caches_are_refused(lib, name, kw):
    assert CALLS[name](lib, cache(**kw)) == pkg.ATTN_ERR_INVALID_ARG
    assert getattr(lib, {"append": "attn_cache_append"}.get(name, "attn_cache_append"))(
        None, NK, NV, TABLE, 4, LENS, None, 2, 3, pkg.ATTN_BF16, None) == pkg.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("name,kw", [
    ("append", dict(dtype=pkg.ATTN_BF16_OUT_F32)), ("append", dict(dtype=9)), ("append", dict(S=-1)),
    ("append", dict(B=-1)), ("append", dict(k=None)), ("append", dict(v=NV + 8)), ("append", dict(table=None)),
    ("append", dict(table=TABLE + 2)), ("append", dict(pos=None)), ("append", dict(counts=COUNTS + 1)),
    ("append", dict(max_pages=0)), ("append", dict(max_pages=(2 ** 31 - 1024) // 16)), ("append", dict(k=K)),
    ("append", dict(v=KB)), ("append", dict(table=VS)), ("append", dict(counts=K + 64)), ("append", dict(B=1 << 20, S=1 << 20)),
    ("read", dict(dtype=pkg.ATTN_F16_OUT_F32)), ("read", dict(S=-1)), ("read", dict(k=None)),
    ("read", dict(v=NV + 4)), ("read", dict(v=NK + 64)), ("read", dict(k=K)), ("read", dict(v=KS)),
    ("read", dict(k=TABLE)), ("read", dict(lens=None)), ("read", dict(max_pages=-3)),
    ("select", dict(q=None)), ("select", dict(q=Q + 8)), ("select", dict(n=0)), ("select", dict(n=-2)),
    ("select", dict(n=27649)), ("attend", dict(pages=PAGES, n=27649)),
    ("select", dict(H=3)), ("select", dict(H=0)), ("select", dict(H=2 * 129)), ("select", dict(Sq=-1)),
    ("select", dict(causal=2)), ("select", dict(dtype=5)), ("select", dict(pages=None)),
    ("select", dict(pages=PAGES + 2)), ("select", dict(pages=Q)), ("select", dict(ws=None)),
    ("select", dict(ws=WS + 8)), ("select", dict(bytes=2 * 2 * 8 * 4 - 1)), ("select", dict(ws=K)),
    ("select", dict(ws=PAGES)), ("select", dict(max_pages=27649)), ("select", dict(lens=None)),
    ("attend", dict(q=None)), ("attend", dict(o=None)), ("attend", dict(o=O + 8)), ("attend", dict(lse=L + 2)),
    ("attend", dict(H=5)), ("attend", dict(H=-2)), ("attend", dict(max_pages=1 << 30)), ("attend", dict(Sq=-1)), ("attend", dict(B=4097)),
    ("attend", dict(causal=3)), ("attend", dict(scale=float("nan"))), ("attend", dict(scale=float("inf"))),
    ("attend", dict(dtype=-1)), ("attend", dict(n=2)), ("attend", dict(pages=PAGES, n=0)),
    ("attend", dict(pages=PAGES + 1, n=2)), ("attend", dict(ws=None)), ("attend", dict(ws=WS + 4)),
    ("attend", dict(bytes=64)), ("attend", dict(o=Q)), ("attend", dict(o=V)), ("attend", dict(lse=KS)),
    ("attend", dict(lse=O)), ("attend", dict(ws=O)), ("attend", dict(o=TABLE)), ("attend", dict(ws=Q)),
    ("attend", dict(pages=O, n=2)),
], ids=lambda x: x if isinstance(x, str) else ",".join("%s=%s" % i for i in x.items()))
def test_bad_arguments_are_refused(lib, name, kw):
    assert CALLS[name](lib, **kw) == pkg.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(v=K), dict(v=K + 16), dict(k_scale=V), dict(v_scale=KS), dict(v_scale=KS + 4),
                                dict(k_bounds=K), dict(k_bounds=VS)], ids=str)
def test_append_refuses_a_cache_whose_arrays_overlap(lib, kw):
    assert append(lib, cache(**kw)) == pkg.ATTN_ERR_INVALID_ARG


def test_select_needs_bounds(lib):
    assert select(lib, cache(k_bounds=None)) == pkg.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("name,kw", [("append", dict(B=0)), ("append", dict(S=0)), ("read", dict(B=0)),
                                     ("read", dict(S=0)), ("select", dict(B=0)), ("select", dict(Sq=0)),
                                     ("attend", dict(B=0)), ("attend", dict(Sq=0))])
def test_empty_calls_do_nothing(lib, name, kw):
    none = dict.fromkeys({"append": ("k", "v"), "read": ("k", "v"), "select": ("q", "pages", "ws"),
                          "attend": ("q", "o", "lse", "ws")}[name])
    assert CALLS[name](lib, **kw, **none) == pkg.ATTN_OK


def test_workspace_sizes(lib):
    assert pkg.attn_cache_select_workspace_size(2, 3, 4, 10) == (pkg.ATTN_OK, 24 * 80)
    assert pkg.attn_cache_select_workspace_size(0, 3, 4, 10) == (pkg.ATTN_OK, 0)
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, -1, 1), (1, 1, 1, 0), (1, 1, 1, 27649)):
        assert pkg.attn_cache_select_workspace_size(*bad)[0] == pkg.ATTN_ERR_INVALID_ARG
    for args in ((1, 8, 8, 1, 128, 1), (64, 32, 8, 5, 64, 0), (1, 32, 1, 1, 128, 1, 7)):
        st, n = pkg.attn_fwd_cache_workspace_size(*args)
        assert st == pkg.ATTN_OK and n > 0
    for bad in ((1, 8, 3, 1, 128, 1), (1, 8, 8, 1, 96, 1), (1, 8, 8, 1, 128, 7), (4097, 8, 8, 1, 128, 1),
                (1, 8, 8, -1, 128, 1), (1, 8, 8, 1, 128, 1, -1), (1, 0, 1, 1, 128, 1)):
        assert pkg.attn_fwd_cache_workspace_size(*bad)[0] == pkg.ATTN_ERR_INVALID_ARG


def test_status_text(lib):
    assert "table" in pkg.attn_strerror(pkg.ATTN_ERR_TABLE)


def test_cache_class_refuses_what_the_kernels_cannot_take():
    def make(n=4, h=2, page=16, d=64, dtype=torch.int8, **kw):
        t = dict(k=torch.zeros((n, h, page, d), dtype=dtype), v=torch.zeros((n, h, page, d), dtype=dtype),
                 k_scale=torch.zeros(n, h), v_scale=torch.zeros(n, h))
        t.update(kw)
        return pkg.KVCache(**t)

    for kw in (dict(), dict(dtype=torch.uint8), dict(page=24), dict(d=80),
               dict(v=torch.zeros((4, 2, 16, 128), dtype=torch.int8)),
               dict(v=torch.zeros((4, 2, 16, 64), dtype=torch.float8_e4m3fn)),
               dict(k=torch.zeros((4, 2, 16), dtype=torch.int8))):
        with pytest.raises(ValueError):  # the first: not on a CUDA device
            make(**kw)
