"""The wrappers record nothing for autograd, and say so where it would be missed; they give the same bits
without their host side in C++."""
import warnings

import pytest
import torch

import online_softmax_forward_gb300 as pkg
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu


def calls(dt):
    ensure_built()
    new = lambda *s: torch.randn(*s, device="cuda").to(dt)  # noqa: E731
    x = dict(q=new(1, 4, 40, 64), k=new(1, 2, 50, 64), v=new(1, 2, 50, 64))
    o, lse = pkg.attention(**x)
    rot, pos = pkg.Rotary(64), torch.zeros(1, 40, dtype=torch.int32, device="cuda")
    kr = new(1, 2, 40, 64)
    return {
        "attention": (lambda **c: pkg.attention(**{**x, **c}), ("q", "k", "v")),
        "attention_bwd": (lambda **c: pkg.attention_bwd(**{**x, "o": o, "lse": lse, "do": o, **c}),
                          ("q", "k", "v", "o", "lse", "do", "dlse")),
        "rotary": (lambda q=x["q"], k=kr: pkg.rotary(q, k, rot, pos), ("q", "k")),
    }, dict(x, o=o, lse=lse, do=o, dlse=torch.zeros_like(lse), rotary_k=kr)


@pytest.mark.parametrize("name", ["attention", "attention_bwd", "rotary"])
def test_a_gradient_that_is_not_recorded_is_announced(name):
    all_calls, tensors = calls(torch.bfloat16)
    call, args = all_calls[name]
    want = call()
    for arg in args:
        t = tensors["rotary_k" if (name, arg) == ("rotary", "k") else arg]
        leaf = t.detach().clone().requires_grad_()
        with pytest.warns(UserWarning, match="no gradient") as seen:
            got = call(**{arg: leaf})
        assert seen[0].filename == __file__  # points at the call
        assert not any(r.requires_grad for r in got)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.no_grad():
                again = call(**{arg: leaf})
            call(**{arg: leaf.detach()})
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, again))


@pytest.mark.parametrize("name", ["attention_bwd", "rotary"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
def test_without_their_host_side_in_c(name, dt, monkeypatch):
    """The wrappers' Python code alone, as where _torch_calls.so was not built: the same bits."""
    call = calls(dt)[0][name][0]
    want = call()
    monkeypatch.setattr(pkg, "_calls", pkg._NoCalls)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
