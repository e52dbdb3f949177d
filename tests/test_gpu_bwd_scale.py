"""attention_bwd in fp16 where the sequences, heads and rows of one call have gradients of very different
size: dS is held in fp16 under powers of two, and each sum has to get one that fits its own terms."""
import math

import pytest
import torch

import online_softmax_forward_gb300 as pkg
from grad_ref import assert_gradients, backward64, forward64
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

HF, F = torch.float16, torch.float32


def make(B, H, Hkv, Sq, Skv, d, sizes, seed, causal, spread=1.0):
    """``sizes``: |do| of each element, broadcast to [B, H, Sq, 1]."""
    ensure_built()
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = (rnd(B, H, Sq, d) * spread).to(HF), rnd(B, Hkv, Skv, d).to(HF), rnd(B, Hkv, Skv, d).to(HF)
    o, lse = forward64(q, k, v, causal)
    return dict(q=q, k=k, v=v, o=o.float(), lse=lse.float(), do=(rnd(B, H, Sq, d) * sizes).to(HF))


def call(x, causal):
    got = pkg.attention_bwd(*(x[n].cuda() for n in ("q", "k", "v", "o", "lse", "do")), causal=causal)
    assert pkg.attn_check_status(None) == pkg.ATTN_OK
    return [t.cpu() for t in got]


def part(x, b, h):
    """kv head h of sequence b alone, with its query heads."""
    G = x["q"].shape[1] // x["k"].shape[1]
    return {n: t[b:b + 1, h:h + 1] if n in "kv" else t[b:b + 1, h * G:(h + 1) * G] for n, t in x.items()}


def check(x, causal, skip=()):
    """Each kv head's gradients within what the formulas allow of that head alone (their smallest
    term, 2^-37 of a bound, is then of that head's bound)."""
    got = call(x, causal)
    G = x["q"].shape[1] // x["k"].shape[1]
    for b in range(x["q"].shape[0]):
        for h in range(x["k"].shape[1]):
            if (b, h) in skip:
                continue
            want, errors = backward64(**part(x, b, h), causal=causal)
            mine = got[0][b:b + 1, h * G:(h + 1) * G], got[1][b:b + 1, h:h + 1], got[2][b:b + 1, h:h + 1]
            assert_gradients(mine, want, errors)
    return got


SHAPES = [
    # B, H, Hkv, Sq, Skv, d, causal
    (2, 4, 2, 260, 300, 64, True),
    (3, 2, 2, 130, 3000, 128, False),   # weights of 2^-11: what a small scale loses first
    (2, 6, 2, 40, 2600, 64, True),      # heads of a kv head walked as one
    (1, 3, 3, 200, 100, 128, True),     # rows without a key, P in two parts
]


@pytest.mark.parametrize("c", SHAPES, ids=str)
@pytest.mark.parametrize("sizes", [(300.0, 3e-5), (1e-4, 3000.0, 1.0)], ids=str)
def test_each_head_keeps_its_own_precision(c, sizes):
    B, H, Hkv, Sq, Skv, d, causal = c
    n = B * Hkv
    size = torch.tensor([sizes[i % len(sizes)] for i in range(n)]).view(B, Hkv).repeat_interleave(H // Hkv, 1)
    check(make(B, H, Hkv, Sq, Skv, d, size[..., None, None], Sq + Skv, causal), causal)


@pytest.mark.parametrize("where", ["do", "v", "o"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_infinities_and_nan_stay_with_their_head(where, bad):
    """Heads of small gradients beside one that holds an infinity or a NaN."""
    x = make(2, 4, 2, 150, 2100, 64, torch.tensor([0.01, 0.01, 1e-3, 1e-3]).view(1, 4, 1, 1), 3, True)
    x[where][0, 0, 17, 5] = bad
    check(x, True, skip=((0, 0),))


@pytest.mark.parametrize("c", SHAPES, ids=str)
def test_each_row_of_dq_keeps_its_own_precision(c):
    """A loss on a few tokens: rows of do of very different size in one tile."""
    B, H, Hkv, Sq, Skv, d, causal = c
    size = 10.0 ** (torch.arange(Sq) % 7 * 1.4 - 5)  # 1e-5 .. 2500
    x = make(B, H, Hkv, Sq, Skv, d, size.view(1, 1, Sq, 1), Sq, causal)
    dq = call(x, causal)[0]
    check(x, causal)
    G = H // Hkv
    for i in list(range(0, Sq, 23)) + [Sq - 1]:
        sees = min(Skv, i + Skv - Sq + 1) if causal else Skv
        if sees < 1:
            assert (dq[:, :, i] == 0).all()
            continue
        for b in range(B):
            for h in range(H):
                at = slice(i, i + 1)
                one = dict(q=x["q"][b:b + 1, h:h + 1, at], o=x["o"][b:b + 1, h:h + 1, at],
                           lse=x["lse"][b:b + 1, h:h + 1, at], do=x["do"][b:b + 1, h:h + 1, at],
                           k=x["k"][b:b + 1, h // G:h // G + 1, :sees], v=x["v"][b:b + 1, h // G:h // G + 1, :sees])
                want, errors = backward64(**one)
                # the scale goes by the norms of v over the kv head, here at most twice those of the keys seen
                assert_gradients([dq[b:b + 1, h:h + 1, at]], want[:1], errors[:1], ("dq row %d" % i,))


@pytest.mark.parametrize("dt_o", [HF, F], ids=str)
def test_large_walks_and_splits(dt_o):
    """Units cut into splits, each with a power of two of its own, and 16-bit results."""
    x = make(2, 2, 1, 3000, 400, 64, torch.tensor([2000.0, 1e-2]).view(2, 1, 1, 1), 5, True)
    x["o"] = x["o"].to(dt_o)
    check(x, True)
    x = make(2, 2, 2, 5, 9000, 128, torch.tensor([1e-2, 2000.0]).view(1, 2, 1, 1), 6, False)
    x["o"] = x["o"].to(dt_o)
    check(x, False)


def test_replays_go_by_what_they_are_given():
    """Captured with small gradients, replayed with large ones in another head."""
    names = ("q", "k", "v", "o", "lse", "do")
    first, second = (make(2, 4, 2, 150, 700, 64, torch.tensor(s).view(1, 4, 1, 1), 8 + i, True)
                     for i, s in enumerate(((1e-3, 1e-3, 1e-5, 1e-5), (0.1, 0.1, 3000.0, 3000.0))))
    held = {n: first[n].cuda() for n in names}
    g = torch.cuda.CUDAGraph()
    pkg.attention_bwd(*(held[n] for n in names), causal=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = pkg.attention_bwd(*(held[n] for n in names), causal=True)
    for x in (second, first, second):
        for n in names:
            held[n].copy_(x[n])
        g.replay()
        want = call(x, True)
        torch.cuda.synchronize()
        assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))


@pytest.mark.parametrize("c", SHAPES, ids=str)
def test_bounds_checking_build(c):
    B, H, Hkv, Sq, Skv, d, causal = c
    x = make(B, H, Hkv, Sq, Skv, d, torch.tensor([1e-3, 100.0]).repeat(H)[:H].view(1, H, 1, 1), 9, causal)
    want = call(x, causal)
    y = {n: t.cuda() for n, t in x.items()}
    lib, code = pkg.load_checked_library(), pkg.dtype_code(HF, F)
    out = [torch.full(y[n].shape, 7.0, device="cuda") for n in "qkv"]
    st, need = pkg.attn_bwd_workspace_size(B, H, Hkv, Sq, Skv, d, causal, code)
    ws = torch.full((need + 64,), 9, dtype=torch.uint8, device="cuda")
    st = lib.attn_bwd(*(y[n].data_ptr() for n in ("q", "k", "v", "o", "lse", "do")), None,
                      *(t.data_ptr() for t in out), B, H, Hkv, Sq, Skv, d, int(causal), 0.0, code,
                      ws.data_ptr() + 32, need, None)
    assert st == pkg.ATTN_OK and lib.attn_check_status(None) == pkg.ATTN_OK
    assert all(torch.equal(a.cpu(), b) for a, b in zip(out, want))
    assert (ws[:32] == 9).all() and (ws[-32:] == 9).all()


@pytest.mark.parametrize("B,H,Hkv,S,d", [(1, 2, 2, 700, 64), (2, 4, 2, 520, 128)])
def test_keys_that_are_not_seen_do_not_count(B, H, Hkv, S, d):
    """Large values behind a row, in tiles its walk leaves out, cost its dq no precision."""
    x = make(B, H, Hkv, S, S, d, torch.full((1, 1, 1, 1), 1e-2), 11, True)
    x["v"][:, :, 512:] = 6e4
    o, lse = forward64(x["q"], x["k"], x["v"], True)
    x["o"] = o.float()
    dq = call(x, True)[0][:, :, :512]
    seen = {n: t[:, :, :512] for n, t in x.items()}
    for b in range(B):
        for h in range(H):
            one = {n: t[b:b + 1, h * Hkv // H:h * Hkv // H + 1] if n in "kv" else t[b:b + 1, h:h + 1]
                   for n, t in seen.items()}
            want, errors = backward64(**one, causal=True)
            assert_gradients([dq[b:b + 1, h:h + 1]], want[:1], errors[:1], ("dq",))
