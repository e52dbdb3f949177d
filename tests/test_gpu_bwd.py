"""attention_bwd against the 64-bit formulas (tests/grad_ref.py), element by
element: every type and width, shared kv heads, ragged lengths, rows without a
key, an lse that the loss uses, units cut into splits, and the forward pass
with shared kv heads."""
import math

import pytest
import torch

import online_softmax_forward_gb300 as pkg
from grad_ref import assert_gradients, backward64, forward64
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def make(B, H, Hkv, Sq, Skv, d, dt, seed=0, o32=False, dlse=False, causal=False, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = (rnd(B, H, Sq, d) * spread).to(dt), rnd(B, Hkv, Skv, d).to(dt), rnd(B, Hkv, Skv, d).to(dt)
    o, lse = forward64(q, k, v, causal)
    do = (rnd(B, H, Sq, d) * 0.3).to(dt)
    return dict(q=q, k=k, v=v, o=o.to(F if o32 else dt), lse=lse.float(), do=do,
                dlse=rnd(B, H, Sq) * 0.3 if dlse else None)


def call(x, lib=None, **kw):
    ensure_built()
    x = {n: None if t is None else t.cuda() for n, t in x.items()}
    got = pkg.attention_bwd(x["q"], x["k"], x["v"], x["o"], x["lse"], x["do"], dlse=x["dlse"], **kw)
    assert pkg.attn_check_status(None) == pkg.ATTN_OK
    return got


def check(x, causal, scale=None):
    got = call(x, causal=causal, scale=scale)
    want, errors = backward64(**x, causal=causal, scale=scale)
    assert all(t.dtype == x["o"].dtype for t in got)
    assert_gradients(got, want, errors)
    return got


def name(c):
    return "-".join(str(v).replace("torch.", "") for v in c)


CASES = [
    # B, H, Hkv, Sq, Skv, d, causal, type
    (1, 1, 1, 128, 128, 128, False, BF),    # one tile of each
    (1, 1, 1, 128, 128, 64, True, HF),
    (1, 1, 1, 1, 1, 128, True, BF),         # one query, one key
    (1, 2, 1, 1, 300, 64, True, BF),        # one query
    (1, 2, 2, 300, 1, 128, False, HF),      # one key
    (2, 2, 2, 257, 257, 128, True, BF),     # one row behind the last whole tile
    (1, 3, 1, 517, 300, 128, True, BF),     # rows without a key; three heads to one
    (1, 3, 3, 300, 517, 64, True, HF),      # more keys than queries
    (2, 8, 2, 200, 333, 64, False, BF),     # four heads to one
    (1, 5, 1, 640, 640, 128, True, HF),     # five heads to one
    (3, 2, 2, 127, 129, 64, False, BF),
    (1, 4, 4, 1000, 1000, 64, True, BF),
    (1, 40, 40, 300, 300, 128, True, BF),   # more units than SMs
    (1, 8, 2, 77, 900, 128, True, BF),      # few queries: the heads of a kv head share tiles
    (2, 16, 1, 100, 700, 64, True, HF),
    (1, 6, 2, 100, 60, 64, True, BF),       # ... with rows without a key
    (2, 5, 1, 128, 128, 128, True, BF),
    (1, 4, 1, 3, 130, 64, True, F),
    (1, 6, 3, 90, 50, 32, True, F),
    (2, 4, 4, 64, 64, 16, True, F),
    (1, 1, 1, 64, 64, 32, True, F),
    (1, 2, 2, 1, 1, 64, False, F),
    (1, 4, 2, 130, 257, 64, True, F),
    (1, 3, 1, 200, 90, 128, True, F),       # rows without a key
    (2, 6, 2, 33, 500, 16, False, F),
    (1, 2, 1, 500, 31, 32, False, F),
]


@pytest.mark.parametrize("c", CASES, ids=name)
def test_bounds_checking_build(c):
    """Every index and TMA coordinate stays in its buffer, and the gradients are the product's."""
    ensure_built()
    lib = pkg.load_checked_library()
    B, H, Hkv, Sq, Skv, d, causal, dt = c
    x = make(B, H, Hkv, Sq, Skv, d, dt, seed=Sq + 3 * Skv, causal=causal)
    y = {n: t.cuda() for n, t in x.items() if t is not None}
    code = pkg.dtype_code(dt)
    out = [torch.full_like(y[n], 7.0) for n in "qkv"]
    st, need = pkg.attn_bwd_workspace_size(B, H, Hkv, Sq, Skv, d, causal, code)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    st = lib.attn_bwd(*(y[n].data_ptr() for n in ("q", "k", "v", "o", "lse", "do")), None,
                      *(t.data_ptr() for t in out), B, H, Hkv, Sq, Skv, d, int(causal), 0.0, code,
                      ws.data_ptr(), need, None)
    assert st == pkg.ATTN_OK
    assert lib.attn_check_status(None) == pkg.ATTN_OK
    want, errors = backward64(**x, causal=causal)
    assert_gradients(out, want, errors)
    o, lse = torch.empty_like(y["q"]), torch.empty_like(y["lse"])
    st = lib.attn_fwd_gqa(*(t.data_ptr() for t in (y["q"], y["k"], y["v"], o, lse)), B, H, Hkv, Sq, Skv, d,
                          int(causal), 0.0, code, None)
    assert st == pkg.ATTN_OK and lib.attn_check_status(None) == pkg.ATTN_OK
    assert torch.equal(o, pkg.attention(y["q"], y["k"], y["v"], causal=causal)[0])


@pytest.mark.parametrize("c", CASES, ids=name)
def test_gradients(c):
    B, H, Hkv, Sq, Skv, d, causal, dt = c
    check(make(B, H, Hkv, Sq, Skv, d, dt, seed=Sq + 3 * Skv, causal=causal), causal)


@pytest.mark.parametrize("dt,d", [(BF, 128), (HF, 64), (F, 64)], ids=str)
@pytest.mark.parametrize("Sq,Skv,causal,H,Hkv", [
    (1, 9000, False, 2, 2),   # one query row over many key tiles: q units in splits
    (77, 9001, True, 4, 1),
    (5000, 100, False, 4, 1),  # many query tiles of four heads to one key tile: kv units in splits
    (3000, 3000, True, 2, 1),
])
def test_splits(dt, d, Sq, Skv, causal, H, Hkv):
    st, need = pkg.attn_bwd_workspace_size(1, H, Hkv, Sq, Skv, d, causal, pkg.dtype_code(dt))
    fixed = 0 if dt == F else H * -(-Sq // 128) * 128 * 8 + 16384  # row statistics and 15 KB of the rest
    assert st == pkg.ATTN_OK and need > fixed  # partial sums are kept
    check(make(1, H, Hkv, Sq, Skv, d, dt, seed=5, causal=causal), causal)


@pytest.mark.parametrize("dt,d", [(BF, 128), (HF, 64), (F, 32)], ids=str)
def test_lse_gradient_and_scale(dt, d):
    x = make(1, 4, 2, 190, 260, d, dt, seed=8, dlse=True, causal=True)
    check(x, True)
    x = make(1, 2, 2, 140, 150, d, dt, seed=9)
    o, lse = forward64(x["q"], x["k"], x["v"], False, 0.21)
    x["o"], x["lse"] = o.to(dt), lse.float()
    check(x, False, scale=0.21)


@pytest.mark.parametrize("dt", [BF, HF], ids=str)
def test_fp32_gradients_of_16_bit_inputs(dt):
    x = make(2, 4, 2, 300, 200, 128, dt, seed=10, o32=True, causal=True)
    got = check(x, True)
    assert got[0].dtype == F


@pytest.mark.parametrize("H,Hkv,Sq,Skv", [(2, 2, 400, 400), (2, 1, 300, 420), (2, 2, 300, 427), (4, 1, 100, 140),
                                           (3, 1, 128, 129), (2, 2, 600, 300), (2, 1, 140, 128)])
@pytest.mark.parametrize("dt,d", [(BF, 128), (HF, 64), (BF, 64), (HF, 128)])
def test_queries_with_few_keys(dt, d, H, Hkv, Sq, Skv):
    """dS of queries that see up to 128 keys is held to twice 16 bits, and P where there are no more:
    without the outputs' rounding their dq, and dk and dv of calls with no other, come out that close."""
    x = make(1, H, Hkv, Sq, Skv, d, dt, seed=Sq + Skv, o32=True, causal=True)
    check(x, True)
    seen = torch.arange(Sq) + 1 + Skv - Sq
    few = int((seen <= 128).sum())
    want, errors = backward64(**x, causal=True)
    assert few > 0 and (errors[0][:, :, :few] <= 2.0 ** -13 * want[0].abs().amax()).all()
    if Skv <= 128:
        assert all((e <= 2.0 ** -13 * w.abs().amax()).all() for e, w in zip(errors, want))


@pytest.mark.parametrize("size", [1e-7, 1e-4, 300.0])
def test_fp16_follows_the_size_of_do(size):
    """Gradients of a loss that was scaled down or up: dS would leave fp16's range unscaled."""
    x = make(1, 2, 1, 260, 300, 64, HF, seed=11, o32=True, causal=True)
    x["do"] = (x["do"].float() / 0.3 * size).to(HF)
    check(x, True)


@pytest.mark.parametrize("dt", [BF, HF, F], ids=str)
def test_peaked_and_far_scores(dt):
    """Scores of hundreds: P is 0 or 1 nearly everywhere, lse far from 0 on both sides."""
    x = make(1, 2, 2, 200, 300, 64, dt, seed=12, spread=40.0, causal=True)
    check(x, True)
    x["q"] = x["q"] * 0 + 3
    x["k"] = (x["k"] * 0.01 - 4).to(dt)  # every score near -96
    o, lse = forward64(x["q"], x["k"], x["v"], True)
    x["o"], x["lse"] = o.to(dt), lse.float()
    check(x, True)


@pytest.mark.parametrize("dt,d", [(BF, 128), (HF, 64), (F, 32)], ids=str)
def test_empty_rows_do_not_count(dt, d):
    """Rows without a key: whatever o, do and dlse hold there changes nothing."""
    x = make(1, 2, 1, 400, 100, d, dt, seed=13, dlse=True, causal=True)
    base = check(x, True)
    assert (x["lse"][:, :, :300] == -math.inf).all()
    x["o"][:, :, :300], x["do"][:, :, :300], x["dlse"][:, :, :300] = 7.0, 9.0, 5.0
    got = call(x, causal=True)
    assert (got[0][:, :, :300] == 0).all()
    assert all(torch.equal(a, b) for a, b in zip(got, base))


@pytest.mark.parametrize("dt", [BF, F], ids=str)
def test_no_queries_and_no_keys(dt):
    z = lambda *s: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    full = lambda *s: torch.full(s, 3.0, dtype=dt, device="cuda")  # noqa: E731
    for Sq, Skv, B in ((0, 5, 2), (5, 0, 2), (0, 0, 2), (5, 5, 0)):
        q, k = z(B, 4, Sq, 64), z(B, 2, Skv, 64)
        lse = torch.zeros(B, 4, Sq, device="cuda")
        out = full(B, 4, Sq, 64), full(B, 2, Skv, 64), full(B, 2, Skv, 64)
        pkg.attention_bwd(q, k, k, q, lse, q, out=out)
        assert all((t == 0).all() for t in out)
    assert pkg.attn_check_status(None) == pkg.ATTN_OK


@pytest.mark.parametrize("dt,d", [(BF, 128), (HF, 64), (F, 64)], ids=str)
def test_against_differences(dt, d):
    """The gradient along random directions is the change of the loss, by central differences of
    the 64-bit forward pass (step h: error h^2 of the third derivative, far below 1 %)."""
    x = make(1, 2, 1, 150, 170, d, dt, seed=14, dlse=True, causal=True)
    got = [t.cpu().double() for t in call(x, causal=True)]
    g = torch.Generator().manual_seed(1)
    h = 1e-3

    def loss(q, k, v):
        o, lse = forward64(q, k, v, True)
        return (o * x["do"].double()).sum() + (lse * x["dlse"].double()).sum()

    args = [x[n].double() for n in "qkv"]
    for i in range(3):
        step = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * step, args[i] - h * step
        want = ((loss(*up) - loss(*down)) / (2 * h)).item()
        have = (got[i] * step).sum().item()
        # the sum of n products with independent errors of u relative to each: 4 u |grad| |step| / sqrt(n)
        u = torch.finfo(dt).eps / 2
        tol = 4 * u * got[i].norm().item() + 1e-4 * (abs(want) + got[i].norm().item())
        assert abs(have - want) <= tol, (i, have, want, tol)


def test_equal_calls_give_equal_bits_and_follow_their_stream():
    x = {n: t.cuda() if t is not None else None
         for n, t in make(2, 8, 2, 700, 900, 128, BF, seed=15, causal=True).items()}
    args = x["q"], x["k"], x["v"], x["o"], x["lse"], x["do"]
    a = pkg.attention_bwd(*args, causal=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = pkg.attention_bwd(*args, causal=True, stream=side)
    with torch.cuda.stream(side):
        c = pkg.attention_bwd(*args, causal=True)
    side.synchronize()
    for s, t, r in zip(a, b, c):
        assert torch.equal(s, t) and torch.equal(s, r)


@pytest.mark.parametrize("dt,d,Sq,Skv", [(BF, 128, 300, 420), (F, 64, 100, 130), (HF, 64, 3, 9000)], ids=str)
def test_captured_and_replayed(dt, d, Sq, Skv):
    xs = [{n: t.cuda() if t is not None else None
           for n, t in make(1, 4, 2, Sq, Skv, d, dt, seed=s, causal=True).items()} for s in (1, 2)]
    names = ("q", "k", "v", "o", "lse", "do")
    held = {n: xs[0][n].clone() for n in names}
    pkg.attention_bwd(*(held[n] for n in names), causal=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = pkg.attention_bwd(*(held[n] for n in names), causal=True)
    for x in xs[::-1]:
        for n in names:
            held[n].copy_(x[n])
        g.replay()
        want = pkg.attention_bwd(*(x[n] for n in names), causal=True)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_key_shards_add_up():
    """dk and dv of a shard of the keys from the merged o and lse; the shards' dq add up."""
    x = {n: t.cuda() if t is not None else None
         for n, t in make(1, 4, 4, 200, 600, 128, BF, seed=16, o32=True).items()}
    q, k, v, do = x["q"], x["k"], x["v"], x["do"]
    parts = [pkg.attention(q, k[:, :, a:a + 200].contiguous(), v[:, :, a:a + 200].contiguous(), out_dtype=F)
             for a in (0, 200, 400)]
    o, lse = pkg.merge(torch.stack([p[0].reshape(-1, 128) for p in parts]),
                       torch.stack([p[1].reshape(-1) for p in parts]))
    o, lse = o.view(q.shape), lse.view(q.shape[:3])
    grads = [pkg.attention_bwd(q, k[:, :, a:a + 200].contiguous(), v[:, :, a:a + 200].contiguous(), o, lse, do)
             for a in (0, 200, 400)]
    got = (sum(g[0] for g in grads), torch.cat([g[1] for g in grads], 2), torch.cat([g[2] for g in grads], 2))
    y = dict(q=q.cpu(), k=k.cpu(), v=v.cpu(), o=o.cpu(), lse=lse.cpu(), do=do.cpu())
    want, errors = backward64(**y)
    assert_gradients(got, want, errors)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last head's gradients are those of that head alone."""
    B, H, Sq, Skv, d = 1, 70000, 130, 250, 128
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB")
    g = torch.Generator(device="cuda").manual_seed(3)
    new = lambda S: torch.randn(B, H, S, d, generator=g, device="cuda", dtype=BF)  # noqa: E731
    q, do, k, v = new(Sq), new(Sq), new(Skv), new(Skv)
    o, lse = pkg.attention(q, k, v, causal=True)
    dq, dk, dv = pkg.attention_bwd(q, k, v, o, lse, do, causal=True)
    for h in (0, 33000, H - 1):
        cut = [t[:, h:h + 1].contiguous() for t in (q, k, v, o, lse, do)]
        alone = pkg.attention_bwd(*cut, causal=True)
        assert all(torch.equal(a[:, h:h + 1], b) for a, b in zip((dq, dk, dv), alone))
    assert pkg.attn_check_status(None) == pkg.ATTN_OK


# ------------------------------------------------------------------ forward with shared kv heads
@pytest.mark.parametrize("c", [
    # B, H, Hkv, Sq, Skv, d, causal, type
    (2, 8, 2, 300, 300, 128, True, BF),
    (1, 6, 1, 517, 300, 64, True, HF),
    (1, 5, 1, 1, 700, 128, False, BF),
    (3, 40, 8, 400, 300, 128, False, BF),
    (2, 4, 2, 130, 257, 64, True, F),      # key-split kernel
    (1, 8, 2, 8, 1024, 32, False, F),      # four warpgroups
    (2, 6, 3, 77, 150, 16, True, F),
    (4, 40, 8, 300, 300, 128, True, F),    # one warpgroup
    (4, 40, 20, 300, 300, 64, True, F),
], ids=name)
def test_shared_heads_equal_repeated_ones(c):
    """Bit for bit the result on k and v with their heads repeated."""
    ensure_built()
    B, H, Hkv, Sq, Skv, d, causal, dt = c
    g = torch.Generator(device="cuda").manual_seed(4)
    new = lambda h, S: torch.randn(B, h, S, d, generator=g, device="cuda").to(dt)  # noqa: E731
    q, k, v = new(H, Sq), new(Hkv, Skv), new(Hkv, Skv)
    o, lse = pkg.attention(q, k, v, causal=causal)
    o2, lse2 = pkg.attention(q, k.repeat_interleave(H // Hkv, 1), v.repeat_interleave(H // Hkv, 1), causal=causal)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o64, lse64 = forward64(q.cpu(), k.cpu(), v.cpu(), causal)
    live = lse64 > -math.inf
    assert (o.cpu().double() - o64).abs().max() <= (1e-5 if dt == F else 2e-2)
    assert (lse.cpu().double() - lse64)[live].abs().max() <= 1e-4
    assert pkg.attn_check_status(None) == pkg.ATTN_OK


# ------------------------------------------------------------------ what callers may do
@pytest.mark.parametrize("dt,d", [(BF, 128), (HF, 64), (F, 64), (F, 16)], ids=str)
def test_sixteen_byte_alignment_and_nothing_beside_the_outputs(dt, d):
    """Inputs and outputs that start 16 bytes behind a 32-byte boundary, outputs with marked
    memory on both sides."""
    x = make(2, 4, 2, 150, 270, d, dt, seed=20, causal=True)
    want, errors = backward64(**x, causal=True)
    pad = 16 // x["q"].element_size()

    def offset(t):
        buf = torch.full((t.numel() + 3 * pad,), 7.0, dtype=t.dtype, device="cuda")
        view = buf[pad:pad + t.numel()].view(t.shape)
        assert view.data_ptr() % 32 == 16
        return buf, view

    y = {}
    for n in ("q", "k", "v", "o", "do"):
        y[n] = offset(x[n])[1].copy_(x[n])
    outs = [offset(x[n]) for n in "qkv"]
    ws = torch.full((pkg.attn_bwd_workspace_size(2, 4, 2, 150, 270, d, 1, pkg.dtype_code(dt))[1] + 32,), 9,
                    dtype=torch.uint8, device="cuda")
    got = pkg.attention_bwd(y["q"], y["k"], y["v"], y["o"], x["lse"].cuda(), y["do"], causal=True,
                            out=[v for _, v in outs], workspace=ws[16:-16])
    assert_gradients(got, want, errors)
    for buf, view in outs:
        assert (buf[:pad] == 7.0).all() and (buf[pad + view.numel():] == 7.0).all()
    assert (ws[:16] == 9).all() and (ws[-16:] == 9).all()
    assert pkg.attn_check_status(None) == pkg.ATTN_OK


def test_two_streams_and_threads_at_once():
    import threading
    xs = [{n: t.cuda() if t is not None else None
           for n, t in make(1, 8, 2, 900, 1100, 128, BF, seed=s, causal=True).items()} for s in range(4)]
    args = [(x["q"], x["k"], x["v"], x["o"], x["lse"], x["do"]) for x in xs]
    want = [pkg.attention_bwd(*a, causal=True) for a in args]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got[i] = pkg.attention_bwd(*args[i], causal=True)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert pkg.attn_check_status(None) == pkg.ATTN_OK


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    import random
    r = random.Random(seed)
    dt = r.choice([BF, HF, F])
    d = r.choice([16, 32, 64, 128] if dt == F else [64, 128])
    Hkv, G, B = r.choice([1, 2, 3]), r.choice([1, 2, 3, 7]), r.choice([1, 1, 2])
    Sq = r.choice([1, 2, 63, 64, 65, 127, 128, 129, r.randint(1, 700)])
    Skv = r.choice([Sq, 1, 64, 128, 255, r.randint(1, 900)])
    causal = r.random() < 0.6
    check(make(B, Hkv * G, Hkv, Sq, Skv, d, dt, seed=seed, causal=causal, dlse=r.random() < 0.4,
               o32=dt != F and r.random() < 0.3), causal)


def test_wrapper_refusals():
    x = {n: t.cuda() if t is not None else None for n, t in make(1, 4, 2, 40, 50, 64, BF, seed=21).items()}
    base = dict(q=x["q"], k=x["k"], v=x["v"], o=x["o"], lse=x["lse"], do=x["do"])
    pkg.attention_bwd(**base)
    for change in (dict(k=x["k"][:, :, :49]), dict(v=x["v"].half()), dict(do=x["do"].float()), dict(o=x["o"].half()),
                   dict(lse=x["lse"].double()), dict(lse=x["lse"][:, :, :39]), dict(q=x["q"].cpu()),
                   dict(q=x["q"].transpose(1, 2).contiguous().transpose(1, 2)), dict(dlse=x["lse"][:, :3]),
                   dict(out=(x["q"].float(), x["k"].clone(), x["v"].clone())),
                   dict(k=x["k"][:, :1].expand(1, 3, 50, 64).contiguous(), v=x["v"][:, :1].expand(1, 3, 50, 64).contiguous()),
                   dict(workspace=torch.empty(100, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            pkg.attention_bwd(**{**base, **change})
    for change in (dict(out=(x["q"], torch.empty_like(x["k"]), torch.empty_like(x["v"]))),
                   dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(scale=math.nan)):
        with pytest.raises(pkg.AttnError):
            pkg.attention_bwd(**{**base, **change})
    assert pkg.attn_check_status(None) == pkg.ATTN_OK


@pytest.mark.parametrize("dt,o32,Sq,Skv", [(BF, False, 300, 300), (HF, True, 40, 7000), (F, False, 65, 64)], ids=str)
def test_both_ways_through_the_wrapper(dt, o32, Sq, Skv):
    """The host side in C++ takes ordinary calls and gives the bits of the Python one; what it does
    not take, it leaves alone."""
    x = {n: t.cuda() for n, t in make(1, 4, 2, Sq, Skv, 64, dt, seed=22, o32=o32, dlse=True).items()}
    order = ("q", "k", "v", "o", "lse", "do", "dlse")
    fast = lambda **change: pkg._fast().attention_bwd(*({**x, **change}[n] for n in order), True, 0.0)  # noqa: E731
    for dlse in (x["dlse"], None):
        a = fast(dlse=dlse)
        out = tuple(torch.empty_like(x[n], dtype=x["o"].dtype) for n in "qkv")
        b = pkg.attention_bwd(**{**x, "dlse": dlse}, causal=True, out=out)
        assert type(a) is tuple and all(torch.equal(s, t) for s, t in zip(a, b))
    other = HF if dt == F else F
    for change in (dict(q=x["q"].cpu()), dict(k=x["k"][:, :, 1:]), dict(v=x["v"].to(other)), dict(do=x["do"].to(other)),
                   dict(o=x["o"].to(torch.float64)), dict(lse=x["lse"].double()), dict(lse=x["lse"][:, :, 1:]),
                   dict(dlse=x["lse"][:, 1:]), dict(dlse=x["lse"].cpu()), dict(q=x["q"].transpose(1, 2)),
                   dict(lse=None), dict(k=x["k"][:, :1].repeat(1, 3, 1, 1), v=x["v"][:, :1].repeat(1, 3, 1, 1))):
        assert fast(**change) is None
    assert pkg._fast().attention_bwd(*(x[n] for n in order), True, math.nan) == pkg.ATTN_ERR_INVALID_ARG
