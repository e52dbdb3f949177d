"""Host-only checks of the backward pass, of rotary positions and of shared kv
heads: every refusal happens before any CUDA call (the addresses are never
read), and the plan of the backward pass covers every pair of tiles once."""
import ctypes
import math

import pytest
import torch

import online_softmax_forward_gb300 as pkg
from online_softmax_forward_gb300 import build as lib_build

GB = 1 << 30
Q, K, V, O, L, DO, DL, DQ, DK, DV, W = (i * GB for i in range(1, 12))


@pytest.fixture(scope="module", autouse=True)
def lib():
    lib_build.build()
    return pkg.load_library()


def bwd(q=Q, k=K, v=V, o=O, lse=L, do=DO, dlse=DL, dq=DQ, dk=DK, dv=DV, B=2, H=8, H_kv=2, Sq=100,
        Skv=200, d=64, causal=1, scale=0.0, dtype=pkg.ATTN_BF16, ws=W, ws_bytes=GB):
    # raw: True and False are what they are for the caller of the C function
    return pkg.load_library().attn_bwd(q, k, v, o, lse, do, dlse, dq, dk, dv, B, H, H_kv, Sq, Skv, d,
                                       causal, scale, dtype, ws, ws_bytes, None)


BAD = [
    dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(lse=None), dict(do=None),
    dict(dq=None), dict(dk=None), dict(dv=None), dict(ws=None),
    dict(q=Q + 8), dict(do=DO + 2), dict(dk=DK + 8), dict(lse=L + 2), dict(dlse=DL + 1), dict(ws=W + 8),
    dict(dq=Q), dict(dk=DV), dict(dv=K + 64), dict(ws=DO), dict(ws=DQ + 256), dict(dq=L), dict(dk=DL),
    dict(ws_bytes=1000), dict(ws_bytes=0),
    dict(H_kv=0), dict(H_kv=3), dict(H_kv=16), dict(H_kv=-2), dict(H=0), dict(H=-8), dict(B=-1),
    dict(Sq=-1), dict(Skv=-1), dict(d=32), dict(d=96), dict(d=0), dict(dtype=pkg.ATTN_F32, d=24),
    dict(dtype=5), dict(dtype=-1), dict(causal=2), dict(causal=-1), dict(scale=math.nan),
    dict(scale=math.inf), dict(B=1 << 20, H=1 << 12, H_kv=1 << 12),
    dict(B=1 << 15, H=1 << 15, H_kv=1 << 15, Sq=1 << 30, Skv=1 << 30),
    dict(B=1, H=1, H_kv=1, Sq=(1 << 31) - 1, Skv=8), dict(B=1, H=1, H_kv=1, Sq=8, Skv=(1 << 31) - 1000),
]


@pytest.mark.parametrize("kw", BAD, ids=lambda kw: ",".join("%s=%s" % i for i in kw.items()))
def test_bwd_refuses(kw):
    assert bwd(**kw) == pkg.ATTN_ERR_INVALID_ARG


def _no_gpu():
    return not torch.cuda.is_available()


def test_bwd_accepts_what_it_documents():
    if not _no_gpu():
        pytest.skip("valid calls with made-up addresses would launch on this host")
    for dt in range(5):
        for d in ((16, 32, 64, 128) if dt == pkg.ATTN_F32 else (64, 128)):
            assert bwd(dtype=dt, d=d) == pkg.ATTN_ERR_UNSUPPORTED_DEVICE
    assert bwd(dlse=None) == pkg.ATTN_ERR_UNSUPPORTED_DEVICE
    assert bwd(H_kv=8) == bwd(H_kv=1) == pkg.ATTN_ERR_UNSUPPORTED_DEVICE
    # one side empty: the other side's gradients are still written, nothing else is needed
    assert bwd(Sq=0, q=None, o=None, lse=None, do=None, dlse=None, dq=None, ws=None, ws_bytes=0) == \
        pkg.ATTN_ERR_UNSUPPORTED_DEVICE
    assert bwd(Skv=0, k=None, v=None, dk=None, dv=None, ws=None, ws_bytes=0) == pkg.ATTN_ERR_UNSUPPORTED_DEVICE
    assert bwd(B=0, q=None, k=None, v=None, o=None, lse=None, do=None, dq=None, dk=None, dv=None, ws=None) == \
        pkg.ATTN_OK


def test_bwd_workspace_size():
    size = lambda *a: pkg.attn_bwd_workspace_size(*a)  # noqa: E731
    st, n = size(2, 8, 2, 100, 200, 64, 1, pkg.ATTN_BF16)
    assert st == pkg.ATTN_OK and n >= 2 * 8 * 128 * 8 and n % 256 == 0
    assert bwd(ws_bytes=n - 1) == pkg.ATTN_ERR_INVALID_ARG
    for empty in ((0, 8, 2, 100, 200), (2, 8, 2, 0, 200), (2, 8, 2, 100, 0)):
        assert size(*empty, 64, 1, pkg.ATTN_BF16) == (pkg.ATTN_OK, 0)
    for bad in ((2, 8, 3, 100, 200, 64, 1, 1), (2, 0, 1, 100, 200, 64, 1, 1), (2, 8, 2, 100, 200, 80, 1, 1),
                (2, 8, 2, -1, 200, 64, 1, 1), (2, 8, 2, 100, 200, 64, 3, 1), (2, 8, 2, 100, 200, 64, 1, 9)):
        assert size(*bad)[0] == pkg.ATTN_ERR_INVALID_ARG
    assert pkg.load_library().attn_bwd_workspace_size(2, 8, 2, 1, 1, 64, 0, 1, None) == pkg.ATTN_ERR_INVALID_ARG


def gqa(q=Q, k=K, v=V, o=O, lse=L, B=2, H=8, H_kv=2, Sq=100, Skv=200, d=64, causal=0, scale=0.0,
        dtype=pkg.ATTN_BF16):
    return pkg.attn_fwd_gqa(q, k, v, o, lse, B, H, H_kv, Sq, Skv, d, causal, scale, dtype, None)


@pytest.mark.parametrize("kw", [
    dict(H_kv=0), dict(H_kv=3), dict(H_kv=-1), dict(H_kv=16), dict(H=0, H_kv=1), dict(q=None), dict(k=K + 8),
    dict(o=Q), dict(lse=O + 16), dict(d=32), dict(causal=2), dict(scale=math.nan), dict(dtype=9),
    # k and v are as large as their own heads make them, and no larger
    dict(o=K + 2 * 2 * 200 * 64 * 2 - 16),
], ids=lambda kw: ",".join("%s=%s" % i for i in kw.items()))
def test_gqa_refuses(kw):
    assert gqa(**kw) == pkg.ATTN_ERR_INVALID_ARG


def test_gqa_accepts_what_it_documents():
    if not _no_gpu():
        pytest.skip("valid calls with made-up addresses would launch on this host")
    assert gqa() == gqa(H_kv=8) == gqa(H_kv=1) == pkg.ATTN_ERR_UNSUPPORTED_DEVICE
    assert gqa(o=K + 2 * 2 * 200 * 64 * 2) == pkg.ATTN_ERR_UNSUPPORTED_DEVICE
    assert gqa(B=0, q=None, k=None, v=None, o=None, lse=None) == pkg.ATTN_OK


def heads(in_=Q, out=O, H=4, in_stride=(4 * 10 * 64, 10 * 64, 64), out_stride=(4 * 10 * 64, 10 * 64, 64)):
    i3 = ctypes.c_int64 * 3
    return pkg._Heads(in_, out, H, i3(*in_stride), i3(*out_stride))


def rot(q="default", k=None, turns=L, width=64, interleaved=0, amplitude=1.0, transpose=0, pos=W, per_token=1,
        B=2, S=10, d=64, dtype=pkg.ATTN_BF16):
    q = heads() if q == "default" else q
    return pkg.load_library().attn_rotary(q, k, turns, width, interleaved, amplitude, transpose, pos, per_token,
                                          B, S, d, dtype, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(turns=None), dict(pos=None), dict(turns=L + 4), dict(pos=W + 2), dict(width=0),
    dict(width=63), dict(width=66), dict(d=63), dict(d=1026), dict(interleaved=2), dict(transpose=-1),
    dict(amplitude=math.nan), dict(amplitude=math.inf), dict(per_token=2), dict(B=-1), dict(S=-1),
    dict(dtype=pkg.ATTN_BF16_OUT_F32), dict(dtype=7), dict(B=1 << 16, S=1 << 15),
    dict(q=heads(in_=None)), dict(q=heads(out=None)), dict(q=heads(in_=Q + 1)), dict(q=heads(H=-1)),
    dict(q=heads(H=65537)), dict(q=heads(in_stride=(-1, 640, 64))),
    dict(q=heads(out_stride=(2560, 640, 32))),      # rows of the output overlap
    dict(q=heads(out_stride=(2560, 0, 64))),        # heads of the output are one
    dict(q=heads(out_stride=(600, 640, 64))),       # sequences of the output overlap
    dict(q=heads(out=Q, out_stride=(4 * 20 * 64, 20 * 64, 64))),  # in place, but elsewhere
    dict(q=heads(in_stride=(1 << 61, 640, 64))),
    dict(k=heads(in_=K, out=None)),
], ids=str)
def test_rotary_refuses(kw):
    assert rot(**kw) == pkg.ATTN_ERR_INVALID_ARG


def test_rotary_accepts_what_it_documents():
    assert rot(B=0, q=heads(in_=None, out=None)) == rot(S=0, q=heads(in_=None)) == pkg.ATTN_OK
    assert rot(q=heads(H=0, in_=None, out=None), turns=None) == pkg.ATTN_OK
    if not _no_gpu():
        pytest.skip("valid calls with made-up addresses would launch on this host")
    ok = pkg.ATTN_ERR_UNSUPPORTED_DEVICE
    assert rot() == rot(k=heads(K, V, 2)) == rot(width=2) == rot(q=heads(out=Q)) == ok
    assert rot(q=heads(in_stride=(0, 0, 0))) == ok                       # a broadcast input
    assert rot(q=heads(in_=Q + 2, in_stride=(2561, 641, 65))) == ok      # no vector fits
    assert rot(q=heads(out_stride=(8 * 64 * 10, 64, 8 * 64))) == ok      # [B][S][heads][d]
    # a dimension of one row has no stride that matters
    assert rot(S=1, q=heads(out_stride=(4 * 64, 64, 0))) == ok


def test_wrappers_refuse_before_any_call():
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    q, k, lse = z(1, 4, 8, 64), z(1, 2, 8, 64), z(1, 4, 8, t=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.attention_bwd(q, k, k, q, lse, q)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.attention(q, k, k)
    with pytest.raises(ValueError, match="shape"):
        pkg.attention(q, z(1, 3, 8, 64), z(1, 3, 8, 64))
    with pytest.raises(ValueError, match="shape"):
        pkg.attention_splitkv(q, k, k, n_splits=1)
    r = pkg.Rotary(64, device="cpu")
    pos = torch.zeros(1, 8, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkg.rotary(q, k, r, pos)  # not on a GPU
    for bad in (dict(width=63), dict(width=0), dict(width=64, layout="other"), dict(width=64, scaling="more"),
                dict(width=64, scaling="parts"), dict(width=64, scaling="parts", context=100, slow=3, fast=2),
                dict(width=2, scaling="base"), dict(width=64, frequencies=[1.0]), dict(width=64, base=-1.0),
                dict(width=2, frequencies=[math.nan]), dict(width=64, amplitude=math.inf),
                dict(width=2, frequencies=[1.0], scaling="linear"), dict(width=64, factor=0.0)):
        with pytest.raises(ValueError):
            pkg.Rotary(**bad, device="cpu")


def test_rotary_angles_are_exact_fractions_of_a_turn():
    """turns / 2^64 of a turn per position is theta to 2^-65 turns (Machin's formula for pi, 200 bits)."""
    one = 1 << 200

    def arctan_inverse(n):
        term, total, k = one // n, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    r = pkg.Rotary(128, device="cpu")
    for theta, t in zip(r.frequencies, r.turns.tolist()):
        num, den = theta.as_integer_ratio()
        want = num * one * 2 ** 63 // (den * pi)  # floor of theta / (2 pi) * 2^64
        assert (t - want) % 2 ** 64 in (0, 1)
    neg = pkg.Rotary(2, frequencies=[-1.0], device="cpu")
    assert (neg.turns.item() + r.turns[0].item()) % 2 ** 64 == 0


def test_calls_on_host_tensors_are_left_to_the_wrapper():
    q, k, pos = torch.zeros(1, 2, 3, 64), torch.zeros(1, 1, 3, 64), torch.zeros(1, 3, dtype=torch.int32)
    lse, rot = torch.zeros(1, 2, 3), pkg.Rotary(64, device="cpu")
    assert pkg._fast().rotary(q, k, pos, False, *rot._args) is None
    assert pkg._fast().rotary(q, None, pos, False) is None
    assert pkg._fast().attention_bwd(q, k, k, q, lse, q, None, False, 0.0) is None
    with pytest.raises(ValueError):
        pkg.rotary(q, k, rot, pos)
    with pytest.raises(ValueError):
        pkg.attention_bwd(q, k, k, q, lse, q)


def test_one_library_serves_every_call(tmp_path):
    """ATTN_GB300_LIB names the library of all functions, those that the wrappers' host side calls among
    them: a second one in the process would have a status word of its own, which nobody reads."""
    import os
    import shutil
    import subprocess
    import sys
    named = str(tmp_path / "libnamed.so")
    shutil.copy(os.path.join(os.path.dirname(pkg.__file__), "libattn.so"), named)
    code = ("import torch, online_softmax_forward_gb300 as pkg\n"
            "assert pkg.attn_abi_version() == pkg.load_library().attn_abi_version()\n"
            "q = torch.zeros(1, 2, 3, 64)\n"
            "assert pkg._fast().rotary(q, None, torch.zeros(1, 3).int(), False, 0, 64, 0, 1.0, -1) is None\n"
            "print(*sorted({l.split()[-1] for l in open('/proc/self/maps') if 'libattn' in l or 'libnamed' in l}))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       env={**os.environ, "ATTN_GB300_LIB": named},
                       cwd=os.path.dirname(os.path.dirname(pkg.__file__)))
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == [named]


def test_binding_torch_is_seen_whole(monkeypatch):
    """A thread that finds torch bound finds all of it: the name that callers look at comes last."""
    import threading
    names = ("_torch", "_int32", "_float32", "_contiguous", "_raw_stream", "_current_device", "_capturing")
    for name in names:
        monkeypatch.setattr(pkg, name, None)
    monkeypatch.setattr(pkg, "_codes", {})
    inside, go = threading.Event(), threading.Event()
    code = pkg.dtype_code

    def slow(*a):
        inside.set()
        assert go.wait(10)
        return code(*a)

    monkeypatch.setattr(pkg, "dtype_code", slow)
    binding = threading.Thread(target=pkg._bind, args=(torch,))
    binding.start()
    assert inside.wait(10)
    early = pkg._torch  # what another thread's call looks at meanwhile
    go.set()
    binding.join()
    assert early is None
    assert all(getattr(pkg, name) is not None for name in names) and len(pkg._codes) == 5


def many(in_, out, H, row=64, **kw):
    """Heads of a packed [B][S][14 heads][64] tensor, in and out."""
    packed = (10 * 14 * 64, 64, 14 * 64)
    return heads(in_, out, H, in_stride=packed, out_stride=packed)


HEAD = 64 * 2  # bytes of a bf16 head
ROWS = 2 * 4 * 10 * 64 * 2  # of the default tensor


@pytest.mark.parametrize("kw", [
    # one output, two tensors
    dict(q=heads(out=O), k=heads(K, O)),
    dict(q=heads(out=O), k=heads(K, O + ROWS - HEAD)),
    dict(q=heads(out=O), k=heads(K, O - ROWS + HEAD)),
    # packed rows: the other's heads begin one too early, or lie where the next token's do
    dict(q=many(Q, O, 8), k=many(Q + 8 * HEAD, O + 7 * HEAD, 4)),
    dict(q=many(Q, O, 8), k=many(Q + 8 * HEAD, O + 11 * HEAD, 4)),
    dict(q=many(Q, O, 8), k=many(Q + 8 * HEAD, O + 8 * HEAD - 2, 4)),
    # an output over the other tensor's input, or over its own elsewhere
    dict(q=many(Q, Q + 8 * HEAD, 8), k=many(Q + 8 * HEAD, O, 4)),
    dict(q=heads(out=K), k=heads(K, V)),
    dict(q=heads(out=O), k=heads(K, Q)),
    dict(q=heads(out=Q + HEAD)),
    dict(q=many(Q, Q + 2 * HEAD, 8)),
    # contiguous rows over packed ones, either way
    dict(q=many(Q, Q, 8), k=heads(K, Q + 64 * HEAD)),
    dict(q=heads(out=Q + HEAD, in_stride=(10 * 14 * 64, 64, 14 * 64))),
    # other strides in the same place: every second head of one, every third of the other
    dict(q=heads(out=O, out_stride=(10 * 64 * 64, 2 * 64, 64 * 64)),
         k=heads(K, O, out_stride=(10 * 64 * 64, 3 * 64, 64 * 64))),
    # a broadcast input under an output
    dict(q=heads(out=O), k=heads(O + ROWS // 2, V, in_stride=(0, 0, 0))),
    # the positions and the angles
    dict(q=heads(out=W)), dict(q=heads(out=W - ROWS + HEAD)), dict(q=heads(out=L)), dict(q=heads(), k=heads(K, W)),
], ids=str)
def test_rotary_refuses_overlap(kw):
    assert rot(**kw) == pkg.ATTN_ERR_INVALID_ARG


def test_rotary_accepts_neighbours():
    """Outputs and inputs that share a buffer and no element of it."""
    if not _no_gpu():
        pytest.skip("valid calls with made-up addresses would launch on this host")
    ok = pkg.ATTN_ERR_UNSUPPORTED_DEVICE
    for kw in (
        dict(q=heads(out=O), k=heads(K, O + ROWS)), dict(q=heads(out=O), k=heads(K, O - ROWS)),
        dict(q=many(Q, O, 8), k=many(Q + 8 * HEAD, O + 8 * HEAD, 4)),
        dict(q=many(Q, Q, 8), k=many(Q + 8 * HEAD, Q + 8 * HEAD, 4)),        # in place
        dict(q=many(Q, Q + 8 * HEAD, 4), k=many(Q, Q + 12 * HEAD, 2)),       # one input for both
        dict(q=many(Q, O, 8), k=many(Q + 8 * HEAD, O + 10 * HEAD, 4)),
        dict(q=heads(out=O, out_stride=(10 * 64 * 64, 2 * 64, 64 * 64)),     # even and odd heads
             k=heads(K, O + HEAD, out_stride=(10 * 64 * 64, 4 * 64, 64 * 64))),
        dict(q=heads(out=Q, H=1, in_stride=(640, 1, 64), out_stride=(640, 9, 64))),  # one head: its stride does not matter
        dict(q=heads(), k=heads(Q, V)),
        dict(q=heads(), k=heads(V, K, in_stride=(0, 0, 0))),
        dict(q=heads(out=W + 80)), dict(q=heads(out=W - ROWS)), dict(q=heads(out=L + 256)),
    ):
        assert rot(**kw) == ok, kw
    assert rot(q=heads(out=O), k=heads(K, O, H=0)) == ok
    assert rot(q=heads(out=W + 8), per_token=0) == ok  # two positions


def test_rotary_overlap_of_random_layouts():
    """The answer is that of the elements counted one by one."""
    if not _no_gpu():
        pytest.skip("valid calls with made-up addresses would launch on this host")
    import itertools
    import random
    r = random.Random(7)
    B, S, d, answers = 2, 3, 4, []
    base = 3 * GB

    def layout(H, nested):
        """Strides of the dimensions in some order, each at least the span of those inside it."""
        strides, span = [0, 0, 0], d
        for i in r.sample(range(3), 3):
            strides[i] = span + r.choice([0, 0, 0, 1, 4, 8, 20]) if nested else r.choice([0, 1, 4, 8, 12, 24, 40])
            span = strides[i] * ((B, H, S)[i] - 1) + span
        return tuple(strides)

    def elements(start, H, strides):
        return {start + b * strides[0] + h * strides[1] + s * strides[2] + c
                for b, h, s, c in itertools.product(range(B), range(H), range(S), range(d))}

    for _ in range(3000):
        Hq, Hk = r.randint(1, 4), r.randint(1, 3)
        strides = [layout(Hq, False), layout(Hq, True), layout(Hk, False), layout(Hk, True)]
        if r.random() < 0.5:
            strides[1] = strides[3] = layout(max(Hq, Hk), True)  # views of one packed tensor
        starts = [r.randint(0, 30), r.randint(100, 400), r.randint(0, 500), r.randint(0, 400)]
        qi, qo, ki, ko = (elements(s, H, t) for s, H, t in zip(starts, (Hq, Hq, Hk, Hk), strides))
        if len(qo) < Hq * B * S * d or len(ko) < Hk * B * S * d:
            continue
        free = not (qo & (qi | ki | ko) or ko & (qi | ki))
        at = [base + 2 * s for s in starts]
        got = rot(q=heads(at[0], at[1], Hq, strides[0], strides[1]), k=heads(at[2], at[3], Hk, strides[2], strides[3]),
                  width=d, d=d, B=B, S=S)
        assert got == (pkg.ATTN_ERR_UNSUPPORTED_DEVICE if free else pkg.ATTN_ERR_INVALID_ARG), (starts, strides, Hq, Hk)
        answers.append(free)
    assert 200 < sum(answers) < len(answers) - 200


def test_bwd_takes_the_lengths_it_documents():
    """Sq and Skv up to 2^31 - 1024, and shared heads whose rows together pass that."""
    top = 2 ** 31 - 1024
    size = lambda **kw: pkg.attn_bwd_workspace_size(*{**dict(B=1, H=1, H_kv=1, Sq=8, Skv=8, d=16, causal=0,  # noqa: E731
                                                             dtype=pkg.ATTN_F32), **kw}.values())[0]
    for kw in (dict(Sq=top), dict(Skv=top), dict(Sq=top, Skv=top, H=2, H_kv=2), dict(Sq=top, d=128, dtype=pkg.ATTN_BF16),
               dict(Skv=top, d=64, dtype=pkg.ATTN_F16, causal=1), dict(H=4, Sq=2 ** 29 - 256), dict(H=4, Sq=2 ** 29 - 200),
               dict(H=4, Sq=2 ** 29 - 33), dict(H=4, Sq=2 ** 29)):
        assert size(**kw) == pkg.ATTN_OK, kw
    for kw in (dict(Sq=top + 1), dict(Skv=top + 1), dict(H=4, Sq=top + 1)):
        assert size(**kw) == pkg.ATTN_ERR_INVALID_ARG, kw
