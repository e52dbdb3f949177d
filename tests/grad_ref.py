"""Plain 64-bit forms of the backward pass and of rotary positions, with bounds
on what the kernels' roundings may cost, element by element."""
from __future__ import annotations

import math

import torch


def visible(Sq, Skv, causal):
    i = torch.arange(Sq)[:, None]
    j = torch.arange(Skv)[None]
    return (j <= i + Skv - Sq) if causal else torch.ones(Sq, Skv, dtype=torch.bool)


def forward64(q, k, v, causal, scale=None):
    """(o, lse) of q [B,H,Sq,d] over k, v [B,H_kv,Skv,d], in float64."""
    G = q.shape[1] // k.shape[1]
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    s = q.double() @ k.double().repeat_interleave(G, 1).mT * scale
    s = s.masked_fill(~visible(q.shape[2], k.shape[2], causal), -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse > -math.inf, lse, 0.0)[..., None])
    return p @ v.double().repeat_interleave(G, 1), lse


def backward64(q, k, v, o, lse, do, dlse=None, causal=False, scale=None):
    """dq, dk, dv and, for each, the largest error that the kernels' roundings allow.

    u is half a step of the operands of the products (P and dS), 0 for fp32 inputs; dS of queries
    that see at most 128 keys, and P if there are no more, are held in two such parts, which leaves
    u * u.  The other
    terms are fp32 arithmetic: a product's sum over d channels in any order and an exponent of a
    few units in the last place of its largest term, and the sums over rows, all taken as 2^-20 of
    the sum of the terms' magnitudes (16 units; sums of n terms grow with sqrt(n) and stay far
    below that at the sizes tested)."""
    dt = q.dtype
    B, H, Sq, d = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    G = H // Hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    u = 0.0 if dt == torch.float32 else torch.finfo(dt).eps / 2
    f = 2.0 ** -20
    q, k, v, o, do = (t.double() for t in (q, k, v, o, do))
    lse = lse.double()
    K, V = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    seen = visible(Sq, Skv, causal)
    l0 = torch.where(lse > -math.inf, lse, 0.0)[..., None]
    live = seen & (lse > -math.inf)[..., None]
    p = torch.where(live, torch.exp(q @ K.mT * scale - l0), 0.0)
    D = (o * do).sum(-1, keepdim=True)
    if dlse is not None:
        D = D - dlse.double()[..., None]
    dp = do @ V.mT
    ds = p * (dp - D)
    # errors of P (in fp32, and as an operand) and dS, which is made of P in fp32
    e32 = p * f * (1 + l0.abs() + scale * (q.abs() @ K.abs().mT))
    us = torch.where(seen.sum(-1, keepdim=True) <= 128, u * u, u)
    ep = p * (u * u if Skv <= 128 else u) + e32
    mag = do.abs() @ V.abs().mT + (o.abs() * do.abs()).sum(-1, keepdim=True)
    if dlse is not None:
        mag = mag + dlse.double().abs()[..., None]
    es = ds.abs() * us + p * f * mag + e32 * (dp - D).abs()
    if dt == torch.float16:
        # floors of fp16 under the scales: P times 2^14; dS brought to at least 2^12 of its bound
        bound = do.norm(dim=-1).amax() * v.norm(dim=-1).amax() + D.abs().amax()
        ep = ep + 2.0 ** -39 * seen
        es = es + 2.0 ** -37 * bound * seen

    def fold(x):  # summed over the query heads of a kv head
        return x.reshape(B, Hkv, G, *x.shape[2:]).sum(2)

    dq, dk, dv = ds @ K * scale, fold(ds.mT @ q) * scale, fold(p.mT @ do)
    eq = (es @ K.abs() + f * (ds.abs() @ K.abs())) * scale
    ek = fold(es.mT @ q.abs() + f * (ds.abs().mT @ q.abs())) * scale
    ev = fold(ep.mT @ do.abs() + f * (p.mT @ do.abs()))
    return (dq, dk, dv), (eq, ek, ev)


def assert_gradients(got, want, errors, names=("dq", "dk", "dv")):
    """|got - want| within the errors plus the output's own rounding."""
    for g, w, e, name in zip(got, want, errors, names):
        t = g.dtype
        out = torch.finfo(t).eps / 2
        tiny = torch.finfo(t).smallest_normal * torch.finfo(t).eps
        g = g.detach().cpu().double()
        assert torch.isfinite(g).all(), name
        allowed = e * (1 + out) + w.abs() * out + tiny + 1e-30
        excess = (g - w).abs() / allowed
        worst = excess.max().item() if excess.numel() else 0.0
        assert worst <= 1.0, "%s: %.2f of the allowed error" % (name, worst)


def rotary64(x, pos, theta, layout="half", amplitude=1.0, transpose=False):
    """x [B,H,S,d] turned by pos [B,S] * theta [n], in float64."""
    n = theta.numel()
    a = pos.double()[:, None, :, None] * theta.double()
    c, s = torch.cos(a) * amplitude, torch.sin(a) * amplitude
    s = -s if transpose else s
    y = x.double().clone()
    if layout == "half":
        i, j = slice(0, n), slice(n, 2 * n)
    else:
        i, j = slice(0, 2 * n, 2), slice(1, 2 * n, 2)
    u, v = x.double()[..., i], x.double()[..., j]
    y[..., i], y[..., j] = u * c - v * s, u * s + v * c
    return y
