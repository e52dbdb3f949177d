"""The paged 8-bit cache in plain fp64 numpy / torch on the CPU, from its
definition (include/attn.h): one page at a time, one row at a time.  Pools are
dicts of numpy arrays: k, v (codes as numbers, fp64), k_scale, v_scale,
k_bounds."""
from __future__ import annotations

import math

import numpy as np
import torch

TOP = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def pow2_scale(amax, fmt):
    if not math.isfinite(amax):
        return math.nan
    if amax == 0.0:
        return 0.0
    e = -126
    while amax > TOP[fmt] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def grid(y, fmt):
    """y rounded to the nearest code, ties to even."""
    if fmt == "int8":
        return np.rint(y)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    return np.rint(y / step) * step


def numbers(codes):
    """Codes of a torch tensor as fp64 numbers."""
    return codes.detach().cpu().to(torch.float32).double().numpy()


def snapshot(cache):
    """A KVCache's tensors as the arrays this module works on."""
    return dict(k=numbers(cache.k), v=numbers(cache.v), k_scale=numbers(cache.k_scale),
                v_scale=numbers(cache.v_scale),
                k_bounds=None if cache.k_bounds is None else numbers(cache.k_bounds))


def append(pool, k, v, table, pos, counts, fmt):
    """Changes the arrays of ``pool`` as attn_cache_append does."""
    page = pool["k"].shape[2]
    for b in range(k.shape[0]):
        for name, x in (("k", k), ("v", v)):
            for h in range(k.shape[1]):
                at = pos[b]
                while at < pos[b] + counts[b]:
                    p, r0 = table[b][at // page], at % page
                    n = min(page - r0, pos[b] + counts[b] - at)
                    rows = x[b, h, at - pos[b]: at - pos[b] + n]
                    old = pool[name + "_scale"][p, h] if r0 else 0.0
                    now = pow2_scale(np.abs(rows).max() if np.isfinite(rows).all() else math.nan, fmt)
                    now = math.nan if math.isnan(old) or math.isnan(now) else max(old, now)
                    put = lambda y: grid(y / now, fmt) if now > 0 else np.zeros_like(y)  # noqa: E731
                    codes = pool[name][p, h]
                    if r0 and not now == old:
                        codes[:r0] = put(codes[:r0] * old)
                    codes[r0: r0 + n] = put(rows)
                    pool[name + "_scale"][p, h] = now
                    if name == "k" and pool["k_bounds"] is not None:
                        edge = pool["k_bounds"][p, h]
                        lo, hi = codes[r0: r0 + n].min(0), codes[r0: r0 + n].max(0)
                        if r0:
                            was = edge if now == old else put(edge * old)
                            lo, hi = np.minimum(lo, was[0]), np.maximum(hi, was[1])
                        edge[0], edge[1] = lo, hi
                    at += n


def read(pool, table, lens, S):
    page, (_, H, _, d) = pool["k"].shape[2], pool["k"].shape
    out = []
    for name in ("k", "v"):
        x = np.zeros((len(lens), H, S, d))
        for b, n in enumerate(lens):
            for j in range(min(n, S)):
                p = table[b][j // page]
                x[b, :, j] = pool[name][p, :, j % page] * pool[name + "_scale"][p][:, None]
        out.append(x)
    return out


def visible(n, cnt, i, causal):
    if i >= cnt:
        return 0
    return min(max(n - cnt + i + 1, 0), n) if causal else n


def select(q, pool, table, lens, counts, n_select, causal):
    B, H, Sq, _ = q.shape
    page, Hkv = pool["k"].shape[2], pool["k"].shape[1]
    G = H // Hkv
    out = np.full((B, Hkv, Sq, n_select), -1, dtype=np.int64)
    for b in range(B):
        for h in range(Hkv):
            for i in range(Sq):
                vis = -(-visible(lens[b], counts[b], i, causal) // page)
                if vis == 0:
                    continue
                score = []
                for p in range(vis - 1):
                    ph = table[b][p]
                    lo, hi = pool["k_bounds"][ph, h] * pool["k_scale"][ph, h]
                    x = q[b, h * G: (h + 1) * G, i]
                    s = np.maximum(x * lo, x * hi).sum(-1).max()
                    score.append(math.inf if math.isnan(s) else s)
                best = sorted(range(vis - 1), key=lambda p: (-score[p], p))[: n_select - 1]
                best = sorted(best + [vis - 1])
                out[b, h, i, : len(best)] = best
    return out


def attention(q, pool, table, lens, counts, causal, scale=None, pages=None):
    """(o, lse, a, vmax): also the largest sum_c |q_c k_c| * scale over the visible keys and the
    largest |v|, which the tolerances are made of."""
    B, H, Sq, d = q.shape
    page, Hkv = pool["k"].shape[2], pool["k"].shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, lse = np.zeros(q.shape), np.full((B, H, Sq), -np.inf)
    most, vmax = 0.0, 0.0
    for b in range(B):
        k, v = read(pool, [table[b]], [lens[b]], lens[b])
        for h in range(H):
            kk, vv = k[0, h // (H // Hkv)], v[0, h // (H // Hkv)]
            for i in range(Sq):
                keys = np.arange(visible(lens[b], counts[b], i, causal))
                if pages is not None:
                    listed = pages[b, h // (H // Hkv), i]
                    keys = np.concatenate([keys[p * page: (p + 1) * page] for p in listed if p >= 0]
                                          or [keys[:0]])
                if not len(keys):
                    continue
                s = kk[keys] @ q[b, h, i] * scale
                most = max(most, (np.abs(kk[keys]) @ np.abs(q[b, h, i]) * scale).max())
                vmax = max(vmax, np.abs(vv[keys]).max())
                m = s.max()
                w = np.exp(s - m)
                o[b, h, i] = w @ vv[keys] / w.sum()
                lse[b, h, i] = m + math.log(w.sum())
    return o, lse, most, vmax
