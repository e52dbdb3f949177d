"""Timed cases of the paged 8-bit key/value cache: quantising it as it is
written, reading it back, attention over it, and attention over the pages a
cheap score selects.

The cache is a pool of pages.  A page holds `page` tokens of every kv head as
8-bit codes (e4m3 or int8), with one scale for each page and kv head; the
value a code stands for is code * scale.  A scale is the smallest power of two
(at least 2^-126) that keeps the page's largest magnitude within the format's
largest code.  A block table gives the pages of each sequence in order.  For
the page score the pool also holds, for each page, kv head and channel, the
smallest and the largest key code.

Where `own` is false, run() computes the operators in elementary torch
operations in 32 bits (page scores in 64, where near ties decide what is
selected); where it is true it makes the calls of the package.
"""
import math

import torch

own = False

FORMATS = {"e4m3": 448.0, "int8": 127.0}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step of 32 sequences writes its new token: the smallest call, latency counts
        dict(name="append_1tok_b32", kind="append", fmt="e4m3", B=32, Hkv=8, d=128, page=64, S=1,
             lo=130, hi=2000, dtype="bf16"),
        # the keys and values of two whole prompts of the 8192-token, 32-head workload
        dict(name="append_prompt_8k", kind="append", fmt="e4m3", B=2, Hkv=32, d=128, page=64, S=8192,
             lo=0, hi=0, dtype="bf16"),
        # a ragged prompt chunk goes in behind what is held, and the whole context comes back in
        # 16 bits, as before a 16-bit attention over it
        dict(name="append_read_chunk_i8", kind="roundtrip", fmt="int8", B=5, Hkv=4, d=64, page=32, S=700,
             lo=0, hi=1333, dtype="fp16"),
        # four long contexts handed to another stage in bf16
        dict(name="read_32k_bf16", kind="read", fmt="e4m3", B=4, Hkv=8, d=128, page=64, S=32768,
             lo=32000, hi=32768, out="bf16"),
        # a few short ragged sequences read for inspection in fp32
        dict(name="read_short_fp32", kind="read", fmt="int8", B=7, Hkv=4, d=128, page=16, S=300,
             lo=1, hi=300, out="fp32"),
        # a single request's decode step: latency
        dict(name="decode_b1_1k", kind="attend", fmt="e4m3", B=1, H=32, Hkv=8, d=128, page=64, Sq=1,
             lo=1000, hi=1000, dtype="bf16", causal=True),
        # the 4 x 32-head, 32768-key decode, one kv head for each query head
        dict(name="decode_b4_h32_32k", kind="attend", fmt="e4m3", B=4, H=32, Hkv=32, d=128, page=64, Sq=1,
             lo=32768, hi=32768, dtype="bf16", causal=False),
        # a serving batch of ragged lengths with grouped heads
        dict(name="decode_b64_ragged_i8", kind="attend", fmt="int8", B=64, H=32, Hkv=8, d=128, page=32, Sq=1,
             lo=200, hi=8192, dtype="fp16", causal=True, empty=True),
        # five draft tokens of each sequence checked at once
        dict(name="verify_5tok_d64", kind="attend", fmt="e4m3", B=16, H=32, Hkv=8, d=64, page=64, Sq=5,
             lo=777, hi=4096, dtype="bf16", causal=True, ragged_q=True),
        # a prompt chunk against the context held so far
        dict(name="chunk_256_of_4k", kind="attend", fmt="e4m3", B=2, H=32, Hkv=8, d=128, page=128, Sq=256,
             lo=4000, hi=4096, dtype="bf16", causal=True),
        # decode over the 32 pages that score highest of 512
        dict(name="sparse_b8_32k", kind="sparse", fmt="e4m3", B=8, H=32, Hkv=8, d=128, page=64, Sq=1,
             lo=20000, hi=32768, n=32, dtype="bf16", causal=True),
        # two tokens of two very long contexts over 96 pages of up to 4096 each
        dict(name="sparse_b2_131k_i8", kind="sparse", fmt="int8", B=2, H=16, Hkv=4, d=128, page=32, Sq=2,
             lo=100000, hi=131072, n=96, dtype="bf16", causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["append", "roundtrip", "read", "attend", "attend", "attend", "sparse"])
    c = dict(kind=kind, fmt=rng.choice(["e4m3", "int8"]), d=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128]), Hkv=rng.choice([1, 2, 3, 4, 8, 16, 32]))
    if kind == "append":
        c["fmt"] = "e4m3"
    if kind in ("append", "roundtrip", "read"):
        S = _log(rng, 1, 8192)
        c["S"] = S
        if kind == "read":
            c["lo"], c["hi"] = rng.randint(0, S), S
        else:
            c["lo"], c["hi"] = 0, rng.randint(0, 2000)
        c["out" if kind == "read" else "dtype"] = rng.choice(list(DTYPES))
        rows = S if kind != "roundtrip" else S + c["hi"]
        c["B"] = _log(rng, 1, max(1, min(64, 32 * 8192 // (rows * c["Hkv"]))))
        return c
    G = rng.choice([1, 2, 4, 5, 8, 16])
    c["Hkv"] = min(c["Hkv"], max(1, 64 // G))
    c["H"] = c["Hkv"] * G
    c["dtype"] = rng.choice(["bf16", "fp16", "bf16", "fp32"])
    c["causal"] = rng.random() < 0.7
    c["ragged_q"] = rng.random() < 0.3
    if kind == "attend":
        c["Sq"] = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 256)])
        c["hi"] = _log(rng, 1, 32768 if c["Sq"] <= 8 else 4096)
        most = 4 * 32 * 32768 if c["Sq"] <= 8 else 2 * 8 * 4096
        c["B"] = _log(rng, 1, max(1, min(64, most // (c["hi"] * c["Hkv"]))))
        c["B"] = max(1, min(c["B"], 2 * 32 * 256 * 4096 // (c["H"] * c["Sq"] * c["hi"])))
        c["lo"] = rng.randint(0, c["hi"])
        return c
    c["Sq"] = rng.choice([1, 1, 2, 3])
    c["page"] = rng.choice([16, 32, 64])
    c["hi"] = _log(rng, 100, 65536)
    c["lo"] = rng.randint(1, c["hi"])
    c["B"] = _log(rng, 1, max(1, min(16, 8 * 8 * 32768 // (c["hi"] * c["Hkv"]))))
    c["n"] = _log(rng, 1, 96)
    return c


def _span(c):
    """The lengths (or positions) of the B sequences: evenly spread, so that their sum is the case's."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    v = [hi - (hi - lo) * b // max(1, B - 1) for b in range(B)]
    if c.get("empty"):
        v[-1] = 0
    return v


def _counts(c, lens):
    """New rows of each sequence, at most what it holds where those rows are queries."""
    n = c.get("Sq", c.get("S"))
    if c["kind"] in ("append", "roundtrip"):
        return [max(0, n - (n // 3) * (b % 3 == 1)) for b in range(c["B"])]
    return [max(0, n - b % 3) if c.get("ragged_q") else n for b in range(c["B"])]


def _pow2_scale(amax, top):
    """The smallest power of two, at least 2^-126, with amax / scale <= top; 0 for amax = 0."""
    m, e = torch.frexp(amax)
    tm, te = math.frexp(top)
    e = (e - te + (m > tm)).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _encode(x, scale, fmt):
    """Codes of x under scale (broadcast), as bytes."""
    y = torch.where(scale > 0, x / torch.where(scale > 0, scale, torch.ones_like(scale)), torch.zeros_like(x))
    if fmt == "e4m3":
        return y.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(y).to(torch.int8).view(torch.uint8)


def _codes(b, fmt):
    """The numbers that the bytes stand for, before their scale."""
    return b.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()


def _typed(b, fmt):
    return b.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    B, Hkv, d, page, fmt = c["B"], c["Hkv"], c["d"], c["page"], c["fmt"]
    span = _span(c)
    counts = _counts(c, span)
    order = torch.randperm(B, generator=g, device=dev)
    held = torch.tensor(span, dtype=torch.int32, device=dev)[order]
    cnt = torch.tensor(counts, dtype=torch.int32, device=dev)[order]
    writes = c["kind"] in ("append", "roundtrip")
    total = held + (cnt if writes else 0)
    most = max(span) + (max(counts) if writes else 0)
    P = max(1, -(-most // page))
    # pages of the pool in random order; the last page belongs to nobody and pads the table
    used = (total + page - 1) // page
    n = B * P + 1
    perm = torch.randperm(n - 1, generator=g, device=dev)[: B * P].view(B, P).to(torch.int32)
    slot = torch.arange(P, device=dev)
    table = torch.where(slot[None, :] < used[:, None], perm, torch.full_like(perm, n - 1)).contiguous()

    def pool(channel):
        x = torch.randn(n, Hkv, page, d, generator=g, device=dev)
        x += 0.7 * torch.randn(n, Hkv, 1, d, generator=g, device=dev)
        x *= channel
        s = _pow2_scale(x.abs().amax((2, 3)), FORMATS[fmt])
        return _encode(x, s[:, :, None, None], fmt), s

    channel = 1 + 3 * (torch.rand(d, generator=g, device=dev) < 0.05).float()
    k, ks = pool(channel)
    v, vs = pool(torch.ones(d, device=dev))
    # smallest and largest key code of the rows held
    fill = torch.zeros(n, dtype=torch.int64, device=dev)
    fill[table.long().flatten()] = (held[:, None].long() - slot * page).clamp(0, page).flatten()
    fill[n - 1] = 0
    live = (torch.arange(page, device=dev) < fill[:, None])[:, None, :, None]
    kc = _codes(k, fmt)
    bounds = torch.stack([torch.where(live, kc, 1e9).amin(2), torch.where(live, kc, -1e9).amax(2)], 2)
    bounds = torch.where(fill[:, None, None, None] > 0, bounds, 0.0)
    kb = _encode(bounds, torch.ones((), device=dev), fmt)
    k[n - 1], v[n - 1], kb[n - 1], ks[n - 1], vs[n - 1] = 0, 0, 0, 0, 0
    del kc, live, bounds
    st = dict(c, k=k, v=v, ks=ks, vs=vs, kb=kb, table=table, lens=held, counts=cnt)
    if writes:
        dt = DTYPES[c["dtype"]]
        x = torch.randn(2, B, Hkv, c["S"], d, generator=g, device=dev)
        st["new_k"], st["new_v"] = (x[0] * channel).to(dt), x[1].to(dt)
        st["total"] = total
    elif c["kind"] != "read":
        x = torch.randn(B, c["H"], c["Sq"], d, generator=g, device=dev)
        st["q"] = x.to(DTYPES[c["dtype"]])
    if own:
        import online_softmax_forward_gb300 as attn
        st["cache"] = attn.KVCache(_typed(k, fmt), _typed(v, fmt), ks, vs, _typed(kb, fmt))
    return st


# ------------------------------------------------------------------ plain forms
def _plain_append(codes, scale, bounds, x, s):
    """Quantises x [B, Hkv, S, d] into the pages of `codes` behind the s["lens"] tokens held; a
    page whose scale has to grow has its older codes rounded again under the new one."""
    fmt, page, S = s["fmt"], s["page"], s["S"]
    pos, cnt, table = s["lens"].long(), s["counts"].long(), s["table"].long()
    B, P = table.shape
    T = (S + page - 2) // page + 1
    lp = pos[:, None] // page + torch.arange(T, device=pos.device)
    there = (lp * page < (pos + cnt)[:, None]) & (cnt > 0)[:, None]
    trash = codes.shape[0] - 1
    phys = torch.where(there, table.gather(1, lp.clamp(max=P - 1)), trash)
    at = lp[:, :, None] * page + torch.arange(page, device=pos.device)       # [B, T, page]
    new = (at >= pos[:, None, None]) & (at < (pos + cnt)[:, None, None]) & there[:, :, None]
    old = (at < pos[:, None, None]) & there[:, :, None]
    row = (at - pos[:, None, None]).clamp(0, S - 1)
    b = torch.arange(B, device=pos.device)[:, None, None]
    fresh = x.permute(0, 2, 1, 3)[b, row].float().permute(0, 1, 3, 2, 4)      # [B, T, Hkv, page, d]
    new_, old_ = new[:, :, None, :, None], old[:, :, None, :, None]
    had = old.any(2)[:, :, None]
    before = torch.where(had, scale[phys], 0.0)                               # [B, T, Hkv]
    kept = codes[phys]
    now = _pow2_scale(torch.where(new_, fresh.abs(), 0.0).amax((3, 4)), FORMATS[fmt])
    now = torch.maximum(before, now)
    value = torch.where(new_, fresh, _codes(kept, fmt) * before[..., None, None])
    coded = _encode(torch.where(new_ | old_, value, 0.0), now[..., None, None], fmt)
    written = torch.where(there[:, :, None, None, None], torch.where(new_ | old_, coded, kept), 0)
    if bounds is not None:
        low = _codes(bounds[phys], fmt) * before[..., None, None]             # [B, T, Hkv, 2, d]
        was = _codes(_encode(low, now[..., None, None], fmt), fmt)
        c = _codes(written, fmt)
        lo = torch.where(new_, c, math.inf).amin(3)
        hi = torch.where(new_, c, -math.inf).amax(3)
        lo = torch.where(had[..., None], torch.minimum(lo, was[:, :, :, 0]), lo)
        hi = torch.where(had[..., None], torch.maximum(hi, was[:, :, :, 1]), hi)
        both = torch.where(there[:, :, None, None, None], torch.stack([lo, hi], 3), 0.0)
        bounds[phys] = _encode(both, torch.ones((), device=both.device), fmt)
    codes[phys] = written
    scale[phys] = torch.where(there[:, :, None], now, 0.0)


def _plain_gather(codes, scale, table, fmt):
    """[B, Hkv, P * page, d] values of the pages of the table."""
    t = table.long()
    x = _codes(codes[t], fmt) * scale[t][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_read(s, lens, out):
    far = torch.finfo(out).max
    S = s["S"] if s["kind"] == "read" else s["table"].shape[1] * s["page"]
    live = (torch.arange(S, device=lens.device) < lens[:, None])[:, None, :, None]
    k = _plain_gather(s["k"], s["ks"], s["table"], s["fmt"])[:, :, :S]
    v = _plain_gather(s["v"], s["vs"], s["table"], s["fmt"])[:, :, :S]
    return (torch.where(live, k, 0.0).clamp(-far, far).to(out),
            torch.where(live, v, 0.0).clamp(-far, far).to(out))


def _limits(s):
    """Keys visible to each query row [B, Sq]."""
    i = torch.arange(s["Sq"], device=s["q"].device)
    lens, cnt = s["lens"].long()[:, None], s["counts"].long()[:, None]
    seen = (lens - cnt + i + 1).clamp(min=0) if s["causal"] else lens.expand(-1, s["Sq"])
    return torch.where(i < cnt, seen, 0)


def _softmax_av(score, seen, v):
    score = torch.where(seen, score, -math.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m > -math.inf, m, 0.0))
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(l > 0, l, 1.0)
    return o, (m + torch.log(l)).squeeze(-1)


def _plain_attend(s):
    B, H, Sq, d = s["q"].shape
    Hkv, page = s["Hkv"], s["page"]
    k = _plain_gather(s["k"], s["ks"], s["table"], s["fmt"])
    v = _plain_gather(s["v"], s["vs"], s["table"], s["fmt"])
    q = s["q"].float().reshape(B, Hkv, -1, d) * (1 / math.sqrt(d))            # group-major rows
    seen = torch.arange(k.shape[2], device=q.device) < _limits(s)[..., None]  # [B, Sq, S]
    seen = seen[:, None].expand(-1, H // Hkv, -1, -1).flatten(1, 2)[:, None]
    o, lse = _softmax_av(q @ k.mT, seen, v)
    return o.reshape(B, H, Sq, d).to(s["q"].dtype), lse.reshape(B, H, Sq)


def _plain_select(s):
    """The n pages of each query and kv head: the page of its last visible key, then those whose
    bound on q . k (from the smallest and largest code of each channel) is highest for any head of
    the group; in ascending order, -1 where there are fewer."""
    B, H, Sq, d = s["q"].shape
    Hkv, n = s["Hkv"], s["n"]
    q = s["q"].double().reshape(B, Hkv, -1, Sq, d)
    t = s["table"].long()
    kb = _codes(s["kb"][t], s["fmt"]).double() * s["ks"][t][..., None, None].double()
    kb = kb.permute(0, 2, 3, 1, 4)[:, :, None]                                # [B, Hkv, 1, 2, P, d]
    bound = q.clamp(min=0) @ kb[:, :, :, 1].mT + q.clamp(max=0) @ kb[:, :, :, 0].mT
    score = bound.amax(2)                                                     # [B, Hkv, Sq, P]
    P = score.shape[-1]
    p = torch.arange(P, device=q.device)
    pages = (_limits(s) + s["page"] - 1) // s["page"]                         # [B, Sq]
    pages = pages[:, None, :, None]
    score = torch.where(p == pages - 1, math.inf, torch.where(p < pages, score, -math.inf))
    top = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]
    top = torch.where(torch.arange(top.shape[-1], device=q.device) < pages, top, P)
    top = torch.nn.functional.pad(top, (0, n - top.shape[-1]), value=P).sort(-1).values
    return torch.where(top < P, top, -1).to(torch.int32)


def _plain_sparse(s):
    B, H, Sq, d = s["q"].shape
    Hkv, page, fmt = s["Hkv"], s["page"], s["fmt"]
    pages = _plain_select(s)                                                  # [B, Hkv, Sq, n]
    b = torch.arange(B, device=pages.device)[:, None, None, None]
    h = torch.arange(Hkv, device=pages.device)[None, :, None, None]
    phys = s["table"].long()[b, pages.long().clamp(min=0)]
    k = (_codes(s["k"][phys, h], fmt) * s["ks"][phys, h][..., None, None]).flatten(3, 4)
    v = (_codes(s["v"][phys, h], fmt) * s["vs"][phys, h][..., None, None]).flatten(3, 4)
    at = pages.long()[..., None] * page + torch.arange(page, device=pages.device)
    seen = (pages[..., None] >= 0) & (at < _limits(s)[:, None, :, None, None])
    seen = seen.flatten(3, 4)[:, :, :, None]                                  # [B, Hkv, Sq, 1, n * page]
    q = s["q"].float().reshape(B, Hkv, -1, Sq, d).transpose(2, 3) * (1 / math.sqrt(d))
    o, lse = _softmax_av(q @ k.mT, seen, v)                                   # [B, Hkv, Sq, G, ...]
    return (pages, o.transpose(2, 3).reshape(B, H, Sq, d).to(s["q"].dtype),
            lse.transpose(2, 3).reshape(B, H, Sq))


def run(s):
    kind, fmt = s["kind"], s["fmt"]
    if own:
        import online_softmax_forward_gb300 as attn
        cache, table, lens, counts = s["cache"], s["table"], s["lens"], s["counts"]
        if kind in ("append", "roundtrip"):
            attn.cache_append(cache, s["new_k"], s["new_v"], table, lens, counts)
            if kind == "roundtrip":
                k, v = attn.cache_read(cache, table, s["total"], table.shape[1] * s["page"],
                                       dtype=s["new_k"].dtype)
                return dict(k=k, v=v, ks=s["ks"], vs=s["vs"])
            return dict(k=cache.k, v=cache.v, ks=s["ks"], vs=s["vs"], kb=cache.k_bounds)
        if kind == "read":
            k, v = attn.cache_read(cache, table, lens, s["S"], dtype=DTYPES[s["out"]])
            return dict(k=k, v=v)
        pages = None
        if kind == "sparse":
            pages = attn.cache_select(s["q"], cache, table, lens, s["n"], counts=counts, causal=s["causal"])
        o, lse = attn.attention_cache(s["q"], cache, table, lens, counts=counts, causal=s["causal"], pages=pages)
        return dict(o=o, lse=lse) if pages is None else dict(pages=pages, o=o, lse=lse)
    if kind in ("append", "roundtrip"):
        _plain_append(s["k"], s["ks"], s["kb"], s["new_k"], s)
        _plain_append(s["v"], s["vs"], None, s["new_v"], s)
        if kind == "roundtrip":
            k, v = _plain_read(s, s["total"], s["new_k"].dtype)
            return dict(k=k, v=v, ks=s["ks"], vs=s["vs"])
        return dict(k=_typed(s["k"], fmt), v=_typed(s["v"], fmt), ks=s["ks"], vs=s["vs"], kb=_typed(s["kb"], fmt))
    if kind == "read":
        k, v = _plain_read(s, s["lens"], DTYPES[s["out"]])
        return dict(k=k, v=v)
    if kind == "attend":
        o, lse = _plain_attend(s)
        return dict(o=o, lse=lse)
    pages, o, lse = _plain_sparse(s)
    return dict(pages=pages, o=o, lse=lse)


# ------------------------------------------------------------------ work
def work(case):
    c = dict(case)
    B, Hkv, d, page = c["B"], c["Hkv"], c["d"], c["page"]
    span = _span(c)
    counts = _counts(c, span)
    size = lambda name: DTYPES[name].itemsize  # noqa: E731
    pages = lambda tokens: -(-tokens // page)  # noqa: E731
    if c["kind"] in ("append", "roundtrip"):
        rows = sum(counts)
        # rows in, codes out, scales and bounds of the touched pages
        touched = sum(pages(p + n) - p // page for p, n in zip(span, counts) if n)
        b = 2 * rows * Hkv * d * (size(c["dtype"]) + 1) + touched * Hkv * (2 * 4 + 2 * d)
        if c["kind"] == "roundtrip":
            P = pages(max(span) + max(counts))
            b += 2 * sum(p + n for p, n in zip(span, counts)) * Hkv * d
            b += 2 * B * Hkv * P * page * d * size(c["dtype"])
        return {"bytes": b, "flops": 4 * rows * Hkv * d}
    if c["kind"] == "read":
        return {"bytes": 2 * Hkv * d * (sum(span) + B * c["S"] * size(c["out"])), "flops": 2 * sum(span) * Hkv * d}
    H, Sq = c["H"], c["Sq"]
    io = 2 * B * H * Sq * d * size(c["dtype"]) + 4 * B * H * Sq
    rows = [(b, max(0, span[b] - counts[b] + i + 1) if c["causal"] else span[b])
            for b in range(B) for i in range(min(Sq, counts[b]))]
    G = H // Hkv
    if c["kind"] == "attend":
        keys = sum(m for _, m in rows)
        return {"bytes": io + 2 * sum(span) * Hkv * (d + 8 / page), "flops": 4 * keys * H * d}
    keys = sum(min(m, c["n"] * page) for _, m in rows)
    scored = sum(pages(m) for m in span)
    return {"bytes": io + 2 * keys * Hkv * d + scored * Hkv * (2 * d + 4),
            "flops": 4 * keys * H * d + 4 * sum(pages(m) for _, m in rows) * Hkv * G * d}


# ------------------------------------------------------------------ 64 bits
def _grid64(y, fmt):
    """y (float64) rounded to the nearest number that a code stands for, ties to even."""
    if fmt == "int8":
        return y.round()
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (y / step).round() * step


def _page64(codes, scale, p, h, fmt):
    b = codes[p, h]
    b = b.view(torch.int8).double() if fmt == "int8" else b.view(torch.float8_e4m3fn).double()
    return b * scale[p, h].double()


def _sequence64(codes, scale, table_row, n, page, fmt):
    """[Hkv, n, d] values of the first n tokens of one sequence."""
    ids = table_row[: -(-n // page)].tolist()
    x = torch.stack([codes[i] for i in ids], 1).flatten(1, 2)[:, :n]
    x = x.view(torch.int8).double() if fmt == "int8" else x.view(torch.float8_e4m3fn).double()
    s = torch.stack([scale[i] for i in ids], 1).double().repeat_interleave(page, 1)[:, :n]
    return x * s[..., None]


def _append64(codes, scale, bounds, x, s):
    """The numbers of the pool's codes, the scales and the bounds after the rows of x are in."""
    fmt, page, top = s["fmt"], s["page"], FORMATS[s["fmt"]]
    value = (codes.view(torch.int8) if fmt == "int8" else codes.view(torch.float8_e4m3fn)).double()
    edge = (bounds.view(torch.int8) if fmt == "int8" else bounds.view(torch.float8_e4m3fn)).double()
    scale = scale.double()
    pos, cnt, table = s["lens"].tolist(), s["counts"].tolist(), s["table"].tolist()
    for b in range(len(pos)):
        at = pos[b]
        while at < pos[b] + cnt[b]:
            r0 = at % page
            r1 = min(page, r0 + pos[b] + cnt[b] - at)
            p = table[b][at // page]
            rows = x[b, :, at - pos[b]: at - pos[b] + r1 - r0].double()       # [Hkv, rows, d]
            amax = rows.abs().amax((1, 2))
            need = torch.exp2(torch.ceil(torch.log2(amax / top)).clamp(min=-126))
            need = torch.where(amax > 0, need, torch.zeros_like(need))
            if r0:
                now = torch.maximum(scale[p], need)
                ratio = (scale[p] / now).nan_to_num(0.0)[:, None, None]
                value[p, :, :r0] = _grid64(value[p, :, :r0] * ratio, fmt)
                lo, hi = _grid64(edge[p] * ratio, fmt).unbind(1)
            else:
                now = need
                lo, hi = torch.full_like(edge[p, :, 0], math.inf), torch.full_like(edge[p, :, 0], -math.inf)
            coded = _grid64((rows / now[:, None, None]).nan_to_num(0.0), fmt)
            value[p, :, r0:r1] = coded
            edge[p] = torch.stack([torch.minimum(lo, coded.amin(1)), torch.maximum(hi, coded.amax(1))], 1)
            scale[p] = now
            at += r1 - r0
    return value, scale, edge


def exact(case, seed):
    s = prepare(case, seed)
    c, kind, fmt, page = dict(case), case["kind"], case["fmt"], case["page"]
    lens, cnt = s["lens"].tolist(), s["counts"].tolist()
    if kind in ("append", "roundtrip"):
        k, ks, kb = _append64(s["k"], s["ks"], s["kb"], s["new_k"], s)
        v, vs, _ = _append64(s["v"], s["vs"], s["kb"], s["new_v"], s)
        if kind == "append":
            return dict(k=k, v=v, ks=ks, vs=vs, kb=kb)
        out = []
        for codes, scale in ((k, ks), (v, vs)):
            x = torch.zeros(c["B"], c["Hkv"], s["table"].shape[1] * page, c["d"], dtype=torch.float64, device="cuda")
            for b, n in enumerate(s["total"].tolist()):
                for j in range(-(-n // page)):
                    p, r = int(s["table"][b, j]), min(page, n - j * page)
                    x[b, :, j * page: j * page + r] = codes[p, :, :r] * scale[p][:, None, None]
            out.append(x)
        return dict(k=out[0], v=out[1], ks=ks, vs=vs)
    if kind == "read":
        out = []
        for codes, scale in ((s["k"], s["ks"]), (s["v"], s["vs"])):
            x = torch.zeros(c["B"], c["Hkv"], c["S"], c["d"], dtype=torch.float64, device="cuda")
            for b, n in enumerate(lens):
                if n:
                    x[b, :, :n] = _sequence64(codes, scale, s["table"][b], n, page, fmt)
            out.append(x)
        return dict(k=out[0], v=out[1])
    B, H, Sq, d = s["q"].shape
    G = H // c["Hkv"]
    o = torch.zeros(B, H, Sq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Sq), -math.inf, dtype=torch.float64, device="cuda")
    picked = torch.full((B, c["Hkv"], Sq, c.get("n", 1)), -1, dtype=torch.int32, device="cuda")
    row = torch.arange(Sq, device="cuda")
    for b, n in enumerate(lens):
        if not n:
            continue
        k = _sequence64(s["k"], s["ks"], s["table"][b], n, page, fmt)
        v = _sequence64(s["v"], s["vs"], s["table"][b], n, page, fmt)
        seen = n - cnt[b] + row + 1 if c["causal"] else torch.full_like(row, n)
        seen = torch.where(row < cnt[b], seen.clamp(min=0), 0)
        if kind == "attend":
            for h in range(H):
                w = (s["q"][b, h].double() @ k[h // G].mT) / math.sqrt(d)
                w = w.masked_fill(torch.arange(n, device="cuda") >= seen[:, None], -math.inf)
                z = torch.logsumexp(w, -1)
                o[b, h] = torch.exp(w - z[:, None]).nan_to_num(0.0) @ v[h // G]
                lse[b, h] = z
            continue
        ids = s["table"][b, : -(-n // page)].long()
        edge = _page64(s["kb"], s["ks"][:, :, None, None], ids, slice(None), fmt)
        for i, m in enumerate(seen.tolist()):
            if not m:
                continue
            for h in range(c["Hkv"]):
                q = s["q"][b, h * G: (h + 1) * G, i].double()
                P = -(-m // page)
                score = torch.maximum(q[:, None] * edge[:P, h, 0], q[:, None] * edge[:P, h, 1]).sum(-1).amax(0)
                score[P - 1] = math.inf
                rank = sorted(range(P), key=lambda j, sc=score.tolist(): (-sc[j], j))[: c["n"]]
                rank = torch.tensor(sorted(rank), device="cuda")
                picked[b, h, i, : len(rank)] = rank.to(torch.int32)
                at = (rank[:, None] * page + torch.arange(page, device="cuda")).flatten()
                at = at[at < m]
                w = (q @ k[h, at].mT) / math.sqrt(d)
                z = torch.logsumexp(w, -1)
                o[b, h * G: (h + 1) * G, i] = torch.exp(w - z[:, None]) @ v[h, at]
                lse[b, h * G: (h + 1) * G, i] = z
    return dict(o=o, lse=lse) if kind == "attend" else dict(pages=picked, o=o, lse=lse)
