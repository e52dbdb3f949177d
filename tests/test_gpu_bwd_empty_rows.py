"""Rows that see no key (lse = -inf): whatever finite numbers o, do and dlse hold there, no gradient of another
row or key changes, and theirs are zero."""
import math

import pytest
import torch

import online_softmax_forward_gb300 as pkg
from grad_ref import forward64
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def make(H, Hkv, Sq, Skv, d, dt, seed):
    ensure_built()
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = rnd(2, H, Sq, d).to(dt), rnd(2, Hkv, Skv, d).to(dt), rnd(2, Hkv, Skv, d).to(dt)
    o, lse = forward64(q, k, v, True)
    x = dict(q=q, k=k, v=v, o=o.float(), lse=lse.float(), do=rnd(2, H, Sq, d).to(dt), dlse=rnd(2, H, Sq))
    return {n: t.cuda() for n, t in x.items()}


def call(x):
    got = pkg.attention_bwd(**x, causal=True)
    assert pkg.attn_check_status(None) == pkg.ATTN_OK
    return got


SHAPES = [
    (2, 1, 400, 100, 128),   # whole tiles of empty rows and one of both kinds
    (3, 3, 150, 70, 64),
    (6, 2, 100, 60, 64),     # heads of a kv head walked as one: empty rows in every tile
    (1, 1, 3000, 200, 64),   # splits
]


@pytest.mark.parametrize("c", SHAPES, ids=str)
@pytest.mark.parametrize("dt,o,do,dlse", [
    (BF, 1e20, 1e20, 1e30),            # o do overflows
    (BF, 1.0, 3.3e38, 0.0),            # do v overflows
    (BF, -3.3e38, 3.3e38, -3.3e38),
    (HF, 1e38, 6e4, 3e38),
    (HF, 0.0, -6e4, 0.0),
    (F, 1e20, 1e20, 1e30),
    (F, -3e38, 3e38, 3e38),
], ids=str)
def test_what_empty_rows_hold_reaches_nothing(c, dt, o, do, dlse):
    H, Hkv, Sq, Skv, d = c
    x = make(H, Hkv, Sq, Skv, d, dt, Sq)
    n = Sq - Skv
    assert (x["lse"][:, :, :n] == -math.inf).all() and (x["lse"][:, :, n:] > -math.inf).all()
    if dt != F:
        x["o"] = x["o"].to(F if abs(o) > 6e4 and dt == HF else dt)
    for name in ("o", "do", "dlse"):
        x[name][:, :, :n] = 0
    base = call(x)
    assert all(t.isfinite().all() for t in base)
    for name, value in (("o", o), ("do", do), ("dlse", dlse)):
        x[name][:, :, :n] = value
        x[name][:, :, :n:2] *= -1  # both signs: sums of infinities would be NaN
        assert x[name].isfinite().all()
    got = call(x)
    assert (got[0][:, :, :n] == 0).all()
    assert all(torch.equal(a, b) for a, b in zip(got, base))
