"""attention_bwd in fp32 at both ends of the range that include/attn.h gives: numbers that the two parts
for the tensor cores still hold."""
import math

import pytest
import torch

import online_softmax_forward_gb300 as pkg
from grad_ref import assert_gradients, backward64, forward64
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

F = torch.float32
TOP = torch.finfo(F).max
BIG = 2.0 ** 128 - 2.0 ** 116 - 2.0 ** 104  # the largest below 2^128 - 2^116, from where numbers count as infinite


def rows(*s, seed):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("H,Sq,Skv,d", [(1, 64, 64, 64), (1, 40, 90, 32), (3, 200, 130, 128), (64, 130, 128, 16)])
@pytest.mark.parametrize("where", ["q", "k", "v", "do"])
@pytest.mark.parametrize("big", [BIG, -BIG, 2.0 ** 127])
def test_largest_numbers(H, Sq, Skv, d, where, big):
    """One number near the top in each head; its partners, and the other gradients, are small enough
    that no sum overflows."""
    ensure_built()
    x = {n: rows(1, H, Sq if n in ("q", "do") else Skv, d, seed=i) for i, n in enumerate(("q", "k", "v", "do"))}
    other = {"q": "k", "k": "q", "v": "do", "do": "v"}[where]
    # +-1 .. 2 times 2^-123 in 8 bits, so that they and their parts are normal numbers
    x[other] = x[other].sign() * (1 + x[other].abs() % 1).bfloat16().float() * 2.0 ** -123
    if where in "qk":
        x["do"] *= 2.0 ** -8
    x[where][0, :, 3, 5] = big
    o, lse = forward64(x["q"], x["k"], x["v"], False)
    # o apart from do: D = rowsum(o do) stays in range, whatever loss such an o belongs to
    x["o"], x["lse"] = rows(1, H, Sq, d, seed=9) * 2.0 ** -123, lse.float()
    got = pkg.attention_bwd(*(x[n].cuda() for n in ("q", "k", "v", "o", "lse", "do")))
    assert pkg.attn_check_status(None) == pkg.ATTN_OK
    want, errors = backward64(**x)
    assert all((w.abs() + e < TOP).all() for w, e in zip(want, errors))
    assert_gradients(got, want, errors)


def test_small_numbers():
    """q of 2^-112 and more beside k that makes up for it."""
    ensure_built()
    x = {n: rows(1, 2, 100, 64, seed=i) for i, n in enumerate(("q", "k", "v", "do"))}
    x["q"] = x["q"].sign() * (2 + x["q"].abs()) * 2.0 ** -113
    x["k"] *= 2.0 ** 111
    o, lse = forward64(x["q"], x["k"], x["v"], False)
    x["o"], x["lse"] = o.float(), lse.float()
    got = pkg.attention_bwd(*(x[n].cuda() for n in ("q", "k", "v", "o", "lse", "do")))
    want, errors = backward64(**x)
    assert_gradients(got, want, errors)


@pytest.mark.parametrize("Sq,Skv,d", [(400, 100, 64), (70, 40, 128)])
def test_empty_rows_may_hold_the_largest_numbers(Sq, Skv, d):
    ensure_built()
    x = {n: rows(1, 2, Sq if n in ("q", "do") else Skv, d, seed=i).cuda() for i, n in enumerate(("q", "k", "v", "do"))}
    x["o"], x["lse"] = pkg.attention(x["q"], x["k"], x["v"], causal=True)
    n = Sq - Skv
    x["do"][:, :, :n] = 0
    base = pkg.attention_bwd(**x, causal=True)
    assert (x["lse"][:, :, :n] == -math.inf).all()
    x["do"][:, :, :n], x["o"][:, :, :n] = TOP, -TOP
    got = pkg.attention_bwd(**x, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(got, base))
