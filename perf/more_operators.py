"""Timed cases of what training an attention layer takes beside the forward
pass: its backward pass, rotary positions with their gradient, and the forward
pass with kv heads that several query heads share.

Backward: from q, do [B, H, Sq, d], k, v [B, Hkv, Skv, d], the forward's o and
lse, and (where a case says so) the gradient dlse of the lse,
    P = exp(scale q k^T - lse) on the visible keys,  D = rowsum(o do) - dlse,
    dS = P (do v^T - D),  dq = scale dS k,  dk = scale dS^T q,  dv = P^T do,
with dk and dv summed over the query heads of a kv head.  Key j is visible to
query i iff j <= i + Skv - Sq where the case is causal.

Rotary: channels (x, y) of pair i at position p become amplitude * (x cos a -
y sin a, x sin a + y cos a) with a = p * theta_i; the pairs of the first `rot`
channels are (i, i + rot / 2) ("half") or (2i, 2i + 1) ("interleaved"), and the
channels behind them stay.  The gradient is the same with -a.

Where `own` is false, run() computes the operators in elementary torch
operations in 32 bits (angles in 64); where it is true it makes the calls of
the package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # a single tile, 64 rows of width 32: the smallest backward pass, latency counts
        dict(name="bwd_tile_fp32", kind="bwd", B=1, H=1, Hkv=1, Sq=64, Skv=64, d=32, dtype="fp32", causal=True, dlse=False),
        # a small layer trained in fp32
        dict(name="bwd_b2_h4_512_fp32", kind="bwd", B=2, H=4, Hkv=4, Sq=512, Skv=512, d=64, dtype="fp32", causal=False, dlse=False),
        # the 8192-token, 32-head causal workload, backwards
        dict(name="bwd_h32_8k_bf16", kind="bwd", B=1, H=32, Hkv=32, Sq=8192, Skv=8192, d=128, dtype="bf16", causal=True, dlse=False),
        # training with four query heads to a kv head at a length that fills no tile
        dict(name="bwd_shared_4001_bf16", kind="bwd", B=2, H=32, Hkv=8, Sq=4001, Skv=4001, d=128, dtype="bf16", causal=True, dlse=False),
        # queries of one sequence over the keys of another, whose lse is used by the loss too
        dict(name="bwd_cross_d64_fp16", kind="bwd", B=3, H=16, Hkv=16, Sq=1000, Skv=2500, d=64, dtype="fp16", causal=False, dlse=True),
        # the last 77 tokens of a long sequence: few query rows, many keys
        dict(name="bwd_77_of_32k_bf16", kind="bwd", B=1, H=32, Hkv=8, Sq=77, Skv=32768, d=128, dtype="bf16", causal=True, dlse=False),
        # one decode step of 32 sequences, each at its own position: latency
        dict(name="rotary_decode_b32", kind="rotary", B=32, H=32, Hkv=8, S=1, d=128, rot=128, layout="half", dtype="bf16",
             packed=True, transpose=False, scaling=None, far=2000),
        # a prompt as the projection leaves it, [token][head][channel], into the attention's layout
        dict(name="rotary_prompt_8k", kind="rotary", B=1, H=32, Hkv=8, S=8192, d=128, rot=128, layout="half", dtype="bf16",
             packed=True, transpose=False, scaling=None, far=0),
        # the gradient of half the channels of a scaled long context, back into the projection's layout
        dict(name="rotary_grad_far_fp16", kind="rotary", B=3, H=24, Hkv=4, S=1537, d=128, rot=64, layout="interleaved", dtype="fp16",
             packed=True, transpose=True, scaling="parts", far=1000000),
        # a small layer in fp32
        dict(name="rotary_b2_h4_512_fp32", kind="rotary", B=2, H=4, Hkv=4, S=512, d=64, rot=64, layout="half", dtype="fp32",
             packed=False, transpose=False, scaling="linear", far=0),
        # the 8192-token causal workload with four query heads to a kv head
        dict(name="fwd_shared_8k_bf16", kind="fwd", B=1, H=32, Hkv=8, Sq=8192, Skv=8192, d=128, dtype="bf16", causal=True),
        # one kv head for all, a ragged chunk behind what was there before
        dict(name="fwd_one_kv_d64_fp16", kind="fwd", B=3, H=16, Hkv=1, Sq=1111, Skv=1777, d=64, dtype="fp16", causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["bwd", "bwd", "bwd", "rotary", "rotary", "fwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    Hkv, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 4, 5, 8])
    c = dict(kind=kind, dtype=dtype, H=Hkv * G, Hkv=Hkv)
    if kind == "rotary":
        c["d"] = rng.choice([64, 128])
        c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2, 32, 24, 10])
        c["S"] = rng.choice([1, _log(rng, 1, 8192)])
        c["B"] = _log(rng, 1, max(1, min(256, 8192 * 40 // (c["S"] * (c["H"] + Hkv)))))
        return dict(c, layout=rng.choice(["half", "interleaved"]), packed=rng.random() < 0.6, transpose=rng.random() < 0.4,
                    scaling=rng.choice([None, None, "linear", "parts"]), far=rng.choice([0, 2000, 100000, 1000000]))
    c["d"] = rng.choice([16, 32, 64, 128] if dtype == "fp32" else [64, 128])
    c["Sq"] = _log(rng, 1, 2048 if dtype == "fp32" else 8192)
    c["Skv"] = c["Sq"] if rng.random() < 0.5 else _log(rng, 1, 4096 if dtype == "fp32" else 32768)
    c["Skv"] = max(2, c["Skv"])  # over a single key the softmax is constant and dq, dk are nothing but rounding
    c["causal"] = rng.random() < 0.6
    # as much work as the largest listed case of the type at most
    most = 64 * 1024 * 1024 if dtype == "fp32" else 32 * 8192 * 8192 // 2
    c["B"] = _log(rng, 1, max(1, min(8, most // (c["H"] * c["Sq"] * c["Skv"]))))
    if c["B"] * c["H"] * c["Sq"] * c["Skv"] > most:
        c["H"], c["Hkv"] = (4, 4) if G == 1 else (4, 2)
        c["Sq"] = min(c["Sq"], max(1, most // (4 * c["Skv"])))
    if kind == "bwd":
        c["dlse"] = rng.random() < 0.25
    return c


# ------------------------------------------------------------------ inputs
def _theta(c):
    """Angles per position of the rot / 2 pairs (float64) and the amplitude."""
    theta = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
    if c["scaling"] is None:
        return theta, 1.0
    f = 8.0
    if c["scaling"] == "linear":
        return theta / f, 1.0
    # by parts: pairs that turn often within the trained context keep their angle, slow ones are
    # stretched, the ones between are blended
    keep = ((4096 * theta / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return theta * (keep + (1 - keep) / f), 1.0 + 0.1 * math.log(f)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["kind"] == "rotary":
        S = c["S"]
        st = dict(c)
        start = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device="cuda")
        st["pos"] = (start + torch.arange(S, device="cuda")).to(torch.int32)
        theta, st["amplitude"] = _theta(c)
        st["theta"] = theta.cuda()
        rows = _normal(g, B, S, H + 2 * Hkv, d).to(dt) if c["packed"] else None
        if c["packed"] and not c["transpose"]:  # queries, keys and values side by side
            st["q"], st["k"] = rows[:, :, :H].transpose(1, 2), rows[:, :, H:H + Hkv].transpose(1, 2)
        else:
            st["q"], st["k"] = _normal(g, B, H, S, d).to(dt), _normal(g, B, Hkv, S, d).to(dt)
        # the gradient goes into its place among the packed rows
        back = c["packed"] and c["transpose"]
        st["out"] = (rows[:, :, :H].transpose(1, 2), rows[:, :, H:H + Hkv].transpose(1, 2)) if back else None
        if own:  # the table of angles that a program keeps
            import online_softmax_forward_gb300 as attn
            st["rotary"] = attn.Rotary(c["rot"], layout=c["layout"], frequencies=theta, amplitude=st["amplitude"])
        return st
    Sq, Skv = c["Sq"], c["Skv"]
    # keys with a common part and some loud channels, as trained layers have them
    loud = 1 + (torch.rand(d, generator=g, device="cuda") < 0.05).float()
    q = _normal(g, B, H, Sq, d).to(dt)
    k = ((_normal(g, B, Hkv, Skv, d) + 0.3 * _normal(g, B, Hkv, 1, d)) * loud).to(dt)
    v = _normal(g, B, Hkv, Skv, d).to(dt)
    st = dict(c, q=q, k=k, v=v)
    if c["kind"] == "bwd":
        st["o"], st["lse"] = _plain_forward(st)
        st["do"] = (0.05 * _normal(g, B, H, Sq, 1).exp() * _normal(g, B, H, Sq, d)).to(dt)
        st["dlse"] = 0.05 * _normal(g, B, H, Sq) if c["dlse"] else None
    return st


# ------------------------------------------------------------------ plain forms
def _grouped(x, Hkv):
    """[B, H, S, d] as [B, Hkv, G * S, d] in 32 bits: the rows that share a kv head."""
    B, H, S, d = x.shape
    return x.float().reshape(B, Hkv, H // Hkv * S, d)


def _seen(s):
    """Visible keys of each query [G * Sq, Skv], or None where all are."""
    if not s["causal"]:
        return None
    i = torch.arange(s["Sq"], device="cuda")[:, None] + (s["Skv"] - s["Sq"])
    seen = torch.arange(s["Skv"], device="cuda") <= i
    return seen.repeat(s["H"] // s["Hkv"], 1)


def _scores(s, seen):
    q, k = _grouped(s["q"], s["Hkv"]), s["k"].float()
    score = (q * (1 / math.sqrt(s["d"]))) @ k.mT
    return score if seen is None else score.masked_fill_(~seen, -math.inf)


def _plain_forward(s):
    B, H, Sq, d = s["q"].shape
    score = _scores(s, _seen(s))
    m = score.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = score.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ s["v"].float()) / torch.where(total > 0, total, 1.0)
    lse = m + torch.log(total)
    return o.reshape(B, H, Sq, d).to(s["q"].dtype), lse.reshape(B, H, Sq)


def _plain_backward(s):
    B, H, Sq, d = s["q"].shape
    Hkv, scale = s["Hkv"], 1 / math.sqrt(d)
    lse = s["lse"].reshape(B, Hkv, -1, 1)
    p = _scores(s, _seen(s)).sub_(torch.where(lse > -math.inf, lse, 0.0)).exp_()
    do = _grouped(s["do"], Hkv)
    dv = p.mT @ do
    delta = (_grouped(s["o"], Hkv) * do).sum(-1, keepdim=True)
    if s["dlse"] is not None:
        delta = delta - s["dlse"].reshape(B, Hkv, -1, 1)
    ds = (do @ s["v"].float().mT).sub_(delta).mul_(p)
    dq = (ds @ s["k"].float()) * scale
    dk = (ds.mT @ _grouped(s["q"], Hkv)) * scale
    t = s["q"].dtype
    return dict(dq=dq.reshape(B, H, Sq, d).to(t), dk=dk.to(t), dv=dv.to(t))


def _plain_rotate(s, x):
    """x [B, h, S, d] with its first `rot` channels turned."""
    rot, half = s["rot"], s["rot"] // 2
    a = s["pos"].double()[:, None, :, None] * s["theta"]
    a = -a if s["transpose"] else a
    cos, sin = (torch.cos(a) * s["amplitude"]).float(), (torch.sin(a) * s["amplitude"]).float()
    y = x.float()
    if s["layout"] == "half":
        a, b = y[..., :half], y[..., half:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos, y[..., rot:]], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        both = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        turned = torch.cat([both, y[..., rot:]], -1)
    return turned.to(x.dtype)


def run(s):
    if own:
        import online_softmax_forward_gb300 as attn
        if s["kind"] == "bwd":
            dq, dk, dv = attn.attention_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], causal=s["causal"], dlse=s["dlse"])
            return dict(dq=dq, dk=dk, dv=dv)
        if s["kind"] == "rotary":
            q, k = attn.rotary(s["q"], s["k"], s["rotary"], s["pos"], transpose=s["transpose"], out=s["out"])
            return dict(q=q, k=k)
        o, lse = attn.attention(s["q"], s["k"], s["v"], causal=s["causal"])
        return dict(o=o, lse=lse)
    if s["kind"] == "bwd":
        return _plain_backward(s)
    if s["kind"] == "rotary":
        q, k = _plain_rotate(s, s["q"]), _plain_rotate(s, s["k"])
        if s["out"] is not None:
            q, k = s["out"][0].copy_(q), s["out"][1].copy_(k)
        return dict(q=q, k=k)
    o, lse = _plain_forward(s)
    return dict(o=o, lse=lse)


# ------------------------------------------------------------------ work
def _pairs(c):
    """Visible (query, key) pairs of one head."""
    Sq, Skv = c["Sq"], c["Skv"]
    if not c["causal"]:
        return Sq * Skv
    first = Skv - Sq + 1  # keys of query 0; the others see one more each
    skip = max(0, 1 - first)
    n = max(0, Sq - skip)
    return n * (first + skip) + n * (n - 1) // 2


def work(case):
    c = dict(case)
    size = DTYPES[c["dtype"]].itemsize
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["kind"] == "rotary":
        rows = B * c["S"] * (H + Hkv)
        return {"bytes": 2 * rows * d * size + 4 * B * c["S"], "flops": 3 * rows * c["rot"]}
    qn, kn, rows = B * H * c["Sq"] * d, B * Hkv * c["Skv"] * d, B * H * c["Sq"]
    if c["kind"] == "fwd":
        return {"bytes": (2 * qn + 2 * kn) * size + 4 * rows, "flops": 4 * _pairs(c) * B * H * d}
    return {"bytes": (4 * qn + 4 * kn) * size + 4 * rows * (2 if c["dlse"] else 1), "flops": 10 * _pairs(c) * B * H * d}


# ------------------------------------------------------------------ 64 bits
def _exact_weights(s, b, h, lse=None):
    """exp(scale q k^T - lse) of one head over its visible keys, and the lse."""
    Sq, Skv = s["Sq"], s["Skv"]
    w = torch.einsum("id,jd->ij", s["q"][b, h].double(), s["k"][b, h * s["Hkv"] // s["H"]].double()) / math.sqrt(s["d"])
    hidden = torch.zeros((), dtype=torch.bool, device="cuda")
    if s["causal"]:
        hidden = torch.ones(Sq, Skv, dtype=torch.bool, device="cuda").triu(Skv - Sq + 1)
        w = w.masked_fill(hidden, -math.inf)
    if lse is None:
        lse = torch.logsumexp(w, 1)
    return torch.exp(w - lse[:, None]).masked_fill(hidden, 0.0), lse


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "rotary":
        out = {}
        angle = s["pos"].double().unsqueeze(-1) * s["theta"]                      # [B, S, rot / 2]
        turn = torch.polar(torch.full_like(angle, s["amplitude"]), -angle if s["transpose"] else angle)
        n = s["rot"] // 2
        for name in ("q", "k"):
            x = s[name].double()
            y = x.clone()
            re = torch.arange(n, device="cuda") * (1 if s["layout"] == "half" else 2)
            im = re + (n if s["layout"] == "half" else 1)
            z = torch.complex(x[..., re], x[..., im]) * turn[:, None]
            y[..., re], y[..., im] = z.real, z.imag
            out[name] = y
        return out
    B, H, Sq, d = s["q"].shape
    q, k, v = s["q"], s["k"], s["v"]
    o, lse = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(B, H, Sq, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(o), torch.zeros(k.shape, dtype=torch.float64, device="cuda"), torch.zeros(k.shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(H):
            e = h * s["Hkv"] // H
            if s["kind"] == "fwd":
                p, lse[b, h] = _exact_weights(s, b, h)
                o[b, h] = p.nan_to_num(0.0) @ v[b, e].double()
                continue
            p, _ = _exact_weights(s, b, h, s["lse"][b, h].double())
            do = s["do"][b, h].double()
            delta = torch.einsum("id,id->i", s["o"][b, h].double(), do)
            if s["dlse"] is not None:
                delta -= s["dlse"][b, h].double()
            ds = p * (do @ v[b, e].double().T - delta[:, None]) / math.sqrt(d)
            dq[b, h] = ds @ k[b, e].double()
            dk[b, e] += ds.T @ q[b, h].double()
            dv[b, e] += p.T @ do
    return dict(o=o, lse=lse) if s["kind"] == "fwd" else dict(dq=dq, dk=dk, dv=dv)
