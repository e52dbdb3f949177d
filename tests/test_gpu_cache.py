"""The paged 8-bit cache on the GPU against its definition in fp64
(cache_ref.py): append, read, page selection and attention, alone and as one
serving loop.

Codes, scales, bounds, page lists and values read back are exact (scales are
powers of two, every rounding is to nearest, ties to even): they are compared
for equality.  Attention is compared within bounds made of

  a     the largest sum_c |q_c k_c| * scale over visible keys: a score is a sum
        of at most 128 exact products, in at most 16 fp32 additions of the
        partial sums (each off by at most 2^-23 of the running magnitude, which
        is at most a), and three fp32 products: e_s = 20 * 2^-23 * a;
  p     weights exp2 (2^-22) kept in 22 bits, or in 11 (16-bit outputs): e_p =
        2^-21, or 2^-21 + 2^-12;
  o     an average of v with weights off by 2 e_s + e_p (numerator and sum) in
        fp32 sums: (2 e_s + 2 e_p + 2^-18) * max|v|, plus half a step of the
        output type times |o| (bf16 2^-9.., as finfo.eps / 2);
  lse   e_s + 2^-20 + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

import cache_ref as ref
import online_softmax_forward_gb300 as pkg
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def status():
    torch.cuda.synchronize()
    return pkg.attn_check_status(None)


def f64(t):
    return t.detach().cpu().double().numpy()


def new_cache(n, h, page, d, fmt, junk=False):
    """A pool whose unwritten parts hold zeros, or every kind of code and scale."""
    ensure_built()
    c = pkg.KVCache.empty(n, h, page, d, dtype=ref.CODE[fmt])
    for t in (c.k, c.v, c.k_bounds):
        u = t.view(torch.uint8)
        if junk:
            g = torch.Generator(device="cuda").manual_seed(9)
            u.copy_(torch.randint(0, 256, u.shape, generator=g, device="cuda").to(torch.uint8))
        else:
            u.zero_()
    for s in (c.k_scale, c.v_scale):
        s.fill_(math.nan if junk else 0.0)
    return c


def tables(lens, page, width, n_pages, seed=0, pad=-1):
    """Each sequence's pages, drawn from the pool without repetition; the rest is padding."""
    rng = np.random.RandomState(seed)
    free = list(rng.permutation(n_pages))
    t = np.full((len(lens), width), pad, dtype=np.int64)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            t[b, j] = free.pop()
    return t


def rows(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    x[..., ::7] *= 5  # a few large channels
    return x.to(dtype)


def filled(lens, H, page, d, fmt, seed=0, width=None, dtype=torch.bfloat16, junk=True):
    """A cache holding random sequences of these lengths: (cache, table, width)."""
    width = width or max(1, max(-(-n // page) for n in lens))
    n_pages = sum(-(-n // page) for n in lens) + 3
    c = new_cache(n_pages, H, page, d, fmt, junk)
    t = tables(lens, page, width, n_pages, seed)
    S = max(max(lens), 1)
    k, v = rows((len(lens), H, S, d), seed + 1, dtype), rows((len(lens), H, S, d), seed + 2, dtype)
    pkg.cache_append(c, k.cuda(), v.cuda(), dev(t), dev([0] * len(lens)), dev(lens))
    assert status() == pkg.ATTN_OK
    return c, t


def same(a, b):
    assert np.array_equal(np.nan_to_num(a, nan=7e9), np.nan_to_num(b, nan=7e9))


def check_pool(c, want):
    got = ref.snapshot(c)
    for name in want:
        if want[name] is not None:
            same(got[name], want[name])


# ------------------------------------------------------------------ append
APPEND = [
    # positions, counts, S, H, d, page
    ([0], [1], 1, 1, 64, 16),
    ([0, 0], [40, 17], 40, 2, 128, 16),
    ([5, 15, 16, 31], [1, 1, 1, 1], 1, 3, 64, 16),        # one token: first, last and inner rows
    ([3, 60, 64, 0], [70, 5, 0, 129], 129, 2, 128, 64),   # a part, none, more than two pages
    ([127, 100], [2, 300], 300, 1, 64, 128),
    ([33, 0, 7], [31, 32, 33], 33, 2, 64, 32),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: "pos%s_n%s_p%d" % (c[0], c[1], c[5]))
def test_append_gives_the_definition(case, dtype, fmt):
    pos, counts, S, H, d, page = case
    B, width = len(pos), max(-(-(p + n) // page) for p, n in zip(pos, counts)) + 1
    n_pages = B * width + 2
    c = new_cache(n_pages, H, page, d, fmt)
    t = tables([p + n for p, n in zip(pos, counts)], page, width, n_pages, seed=4)
    for step, scale in ((0, 0.25), (1, 3.0)):  # what is held, then larger rows: scales grow
        x = [rows((B, H, S if step else max(max(pos), 1), d), 10 + step + i, dtype, scale) for i in (0, 5)]
        at, n = ([0] * B, pos) if step == 0 else (pos, counts)
        before = ref.snapshot(c)
        ref.append(before, f64(x[0]), f64(x[1]), t, at, n, fmt)
        pkg.cache_append(c, x[0].cuda(), x[1].cuda(), dev(t), dev(at), dev(n))
        assert status() == pkg.ATTN_OK
        check_pool(c, before)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_of_special_values(fmt):
    """Zeros, the type's largest and smallest magnitudes, ties and values just off them."""
    d, page = 64, 16
    top = ref.TOP[fmt]
    lines = [
        torch.zeros(d), torch.full((d,), 3.0e38), torch.full((d,), -1e-45), torch.full((d,), 2.0 ** -126),
        torch.arange(d).float() + 0.5, torch.arange(d).float() * top / 63,
        torch.full((d,), top), torch.full((d,), float(np.nextafter(np.float32(top), np.float32(1e9)))),
        torch.linspace(-1, 1, d) * 2.0 ** -9, torch.tensor([1.0625, -1.1875] * (d // 2)),
    ]
    x = torch.stack(lines)[:, None, None]  # one sequence, one page each
    B = x.shape[0]
    c = new_cache(B, 1, page, d, fmt, junk=True)
    t = np.arange(B)[:, None]
    want = ref.snapshot(c)
    ref.append(want, f64(x), f64(-x), t, [0] * B, [1] * B, fmt)
    pkg.cache_append(c, x.cuda(), (-x).cuda(), dev(t), dev([0] * B))
    assert status() == pkg.ATTN_OK
    check_pool(c, want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_row_that_is_not_finite_marks_its_block(fmt, bad):
    d, page = 64, 16
    c = new_cache(4, 2, page, d, fmt)
    t = np.array([[2, 1]])
    x = rows((1, 2, 20, d), 3, torch.float32)
    y = x.clone()
    y[0, 1, 3, 5] = bad  # head 1, first page; values stay finite
    pkg.cache_append(c, y.cuda(), x.cuda(), dev(t), dev([0]))
    want = ref.snapshot(new_cache(4, 2, page, d, fmt))
    ref.append(want, f64(y), f64(x), t, [0], [20], fmt)
    assert status() == pkg.ATTN_OK
    check_pool(c, want)
    k, v = pkg.cache_read(c, dev(t), dev([20]), 20, dtype=torch.float32)
    nan = torch.isnan(k).cpu()
    assert nan[0, 1, :16].all() and not nan[0, 0].any() and not nan[0, 1, 16:].any()
    assert not torch.isnan(v).any()
    # a later token keeps the mark, a page started again loses it
    pkg.cache_append(c, x[:, :, :1].cuda(), x[:, :, :1].cuda(), dev([[2]]), dev([7]))
    assert torch.isnan(c.k_scale[2, 1]) and not torch.isnan(c.k_scale[2, 0])
    pkg.cache_append(c, x[:, :, :1].cuda(), x[:, :, :1].cuda(), dev([[2]]), dev([0]))
    assert not torch.isnan(c.k_scale[2]).any()
    assert status() == pkg.ATTN_OK


def test_append_without_bounds_and_with_default_counts():
    c = new_cache(4, 2, 32, 128, "e4m3")
    bare = pkg.KVCache(c.k.clone(), c.v.clone(), c.k_scale.clone(), c.v_scale.clone())
    x = rows((2, 2, 30, 128), 1, torch.bfloat16).cuda()
    for cc in (c, bare):
        pkg.cache_append(cc, x, -x, dev([[0], [3]]), dev([0, 2]))
    assert status() == pkg.ATTN_OK
    for name in ("k", "v", "k_scale", "v_scale"):
        same(ref.numbers(getattr(c, name)), ref.numbers(getattr(bare, name)))
    with pytest.raises(ValueError):
        pkg.cache_select(x, bare, dev([[0], [3]]), dev([30, 32]), 1)


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", [([1], 1, 1, 64, 16), ([0, 50, 33], 50, 2, 128, 16), ([100, 7], 70, 3, 64, 64),
                                  ([129, 128, 1, 0], 140, 1, 128, 128)], ids=str)
def test_read_gives_what_the_codes_stand_for(case, dtype, fmt):
    lens, S, H, d, page = case
    c, t = filled(lens, H, page, d, fmt)
    k, v = pkg.cache_read(c, dev(t), dev(lens), S, dtype=dtype)
    assert status() == pkg.ATTN_OK
    want = ref.read(ref.snapshot(c), t, lens, S)
    for got, w in zip((k, v), want):
        same(f64(got), f64(torch.from_numpy(w).to(dtype)))


@pytest.mark.parametrize("fmt,x,dtype,far", [
    ("e4m3", 65504.0, torch.float16, 65504.0), ("e4m3", 3.3e38, torch.bfloat16, torch.finfo(torch.bfloat16).max),
    ("e4m3", 3.4e38, torch.float32, torch.finfo(torch.float32).max), ("int8", 65504.0, torch.float16, 65504.0)])
def test_read_clamps_to_the_types_largest_number(fmt, x, dtype, far):
    c = new_cache(1, 1, 16, 64, fmt)
    rows_ = torch.full((1, 1, 2, 64), x)
    rows_[0, 0, 1] *= -1
    pkg.cache_append(c, rows_.cuda(), rows_.cuda(), dev([[0]]), dev([0]))
    k, _ = pkg.cache_read(c, dev([[0]]), dev([2]), 2, dtype=dtype)
    assert status() == pkg.ATTN_OK
    held = np.clip(ref.read(ref.snapshot(c), [[0]], [2], 2)[0], -far, far)
    same(f64(k), f64(torch.from_numpy(held).to(dtype)))
    assert torch.isfinite(k).all()


# ------------------------------------------------------------------ attention
def check_attention(q, c, t, lens, counts, causal, scale=None, out_dtype=None, pages=None, workspace=None):
    o, lse = pkg.attention_cache(q.cuda(), c, dev(t), dev(lens), counts=dev(counts), causal=causal, scale=scale,
                                 out_dtype=out_dtype, pages=None if pages is None else dev(pages),
                                 workspace=workspace)
    assert status() == pkg.ATTN_OK
    o_, lse_, a, vmax = ref.attention(f64(q), ref.snapshot(c), t, lens, counts, causal, scale, pages)
    es = 20 * 2.0 ** -23 * a
    ep = 2.0 ** -21 + (2.0 ** -12 if o.dtype != torch.float32 else 0.0)
    err = np.abs(f64(o) - o_)
    bound = (2 * es + 2 * ep + 2.0 ** -18) * vmax + HALF[o.dtype] * np.abs(o_) * 1.01 + 2.0 ** -24
    assert np.all(err <= bound), "o off by %.3e, bound %.3e" % (err.max(), bound.flat[err.argmax()])
    got = f64(lse)
    none = np.isneginf(lse_)
    assert np.array_equal(np.isneginf(got), none)
    assert np.all(f64(o)[none] == 0)
    lerr = np.abs(got[~none] - lse_[~none])
    assert np.all(lerr <= es + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse_[~none])), "lse off by %.3e" % lerr.max()
    return o, lse


ATTEND = [
    # lens, counts, Sq, H, H_kv, d, page
    ([1], [1], 1, 1, 1, 64, 16),
    ([17], [1], 1, 4, 1, 128, 16),
    ([300, 0, 31, 64], [1, 1, 1, 0], 1, 6, 2, 64, 32),       # an empty sequence, no queries
    ([1000, 129], [1, 1], 1, 8, 8, 128, 64),
    ([500, 33, 7], [5, 2, 5], 5, 4, 2, 128, 64),             # several queries, padded rows
    ([3, 200], [6, 6], 6, 10, 2, 64, 16),                    # fewer tokens than queries: rows without a key
    ([257], [17], 17, 16, 1, 128, 128),                      # many rows, blocks of them
    ([130, 131], [40, 13], 40, 5, 1, 64, 128),
    ([129], [1], 1, 40, 1, 128, 32),                         # 40 heads on one
    ([700, 0, 128, 129], [33, 0, 33, 9], 33, 8, 2, 128, 64), # more than 128 rows, an empty sequence
    ([1100, 64], [20, 20], 20, 4, 2, 64, 16),                # 80 rows: a warp without one
    ([385], [260], 260, 2, 2, 128, 128),                     # causal blocks that end early
    ([50], [60], 60, 3, 1, 64, 32),                          # more queries than tokens
    ([2500], [3], 3, 3, 3, 64, 16),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,out", [(torch.float32, None), (torch.bfloat16, None), (torch.float16, None),
                                       (torch.bfloat16, torch.float32), (torch.float16, torch.float32)],
                         ids=["f32", "bf16", "f16", "bf16_o32", "f16_o32"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "L%s_q%d_H%dx%d_d%d_p%d" % (c[0], c[2], *c[3:]))
def test_attention_over_the_cache(case, dtype, out, causal, fmt):
    lens, counts, Sq, H, Hkv, d, page = case
    c, t = filled(lens, Hkv, page, d, fmt, seed=len(lens) + d)
    check_attention(rows((len(lens), H, Sq, d), 77, dtype), c, t, lens, counts, causal, out_dtype=out)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("factor,scale", [(1e-30, 1e29), (1e30, 1e-31), (50.0, None), (1e-8, 3.0)])
def test_attention_with_large_and_small_magnitudes(fmt, factor, scale):
    """q far outside fp16's range, scores in the hundreds, and almost equal scores."""
    c, t = filled([200, 90], 2, 32, 64, fmt, seed=3)
    q = rows((2, 4, 2, 64), 5, torch.float32) * factor
    check_attention(q, c, t, [200, 90], [2, 2], True, scale=scale)


def test_page_scales_span_many_powers():
    """Pages of very different magnitudes in one sequence, among them one of zeros."""
    page, d = 16, 64
    c = new_cache(8, 1, page, d, "e4m3", junk=True)
    t = np.array([[5, 1, 0, 6, 2]])
    k, v = rows((1, 1, 75, d), 1, torch.float32), rows((1, 1, 75, d), 2, torch.float32)
    for j, f in enumerate((1.0, 1e-20, 0.0, 1e3, 1e-3)):
        k[:, :, j * page: (j + 1) * page] *= min(f, 2.0)
        v[:, :, j * page: (j + 1) * page] *= f
    pkg.cache_append(c, k.cuda(), v.cuda(), dev(t), dev([0]))
    check_attention(rows((1, 3, 1, d), 4, torch.float32), c, t, [75], [1], True)


def test_a_marked_page_shows_in_the_rows_that_see_it_and_in_no_other():
    page, d = 16, 64
    c = new_cache(5, 1, page, d, "e4m3")
    t = np.array([[0, 1, 2]])
    k, v = rows((1, 1, 40, d), 1, torch.float32), rows((1, 1, 40, d), 2, torch.float32)
    v[0, 0, 38, 0] = math.inf  # third page
    pkg.cache_append(c, k.cuda(), v.cuda(), dev(t), dev([0]))
    q = rows((1, 2, 12, d), 3, torch.float32).cuda()  # positions 28 .. 39: four rows see two pages only
    o, lse = pkg.attention_cache(q, c, dev(t), dev([40]))
    assert status() == pkg.ATTN_OK
    assert torch.isfinite(o[:, :, :4]).all() and torch.isnan(o[:, :, 4:]).all()
    assert torch.isfinite(lse).all()  # the keys are fine
    k[0, 0, 38, 0] = math.nan
    pkg.cache_append(c, k.cuda(), k.cuda(), dev(t), dev([0]))
    o, lse = pkg.attention_cache(q, c, dev(t), dev([40]))
    assert torch.isfinite(lse[:, :, :4]).all() and torch.isnan(lse[:, :, 4:]).all()
    # one marked page and nothing else
    o, lse = pkg.attention_cache(q[:, :, :1].contiguous(), c, dev([[2]]), dev([8]))
    assert torch.isnan(lse).all() and torch.isnan(o).all()
    # a query that is not finite spoils its own row only
    q[0, 1, 2, 7] = math.nan
    q[0, 0, 1, 7] = math.inf
    o, _ = pkg.attention_cache(q, c, dev(t), dev([28]), counts=dev([12]))
    fine = torch.isfinite(o).all(-1)[0].cpu()
    assert not fine[1, 2] and not fine[0, 1] and fine.sum() == 22
    assert status() == pkg.ATTN_OK


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Sq", [1, 4, 7, 40])  # the 8-, 16-, 32- and 128-row kernels
def test_references_that_have_to_move(fmt, Sq):
    """Scores that keep growing along the sequence (each stretch far above the last), values whose
    pages grow and shrink by many powers of two, and pages between that nobody weighs: what was
    accumulated has to be carried from one reference to the next."""
    page, d, n = 16, 64, 900
    c = new_cache(60, 1, page, d, fmt, junk=True)
    t = tables([n], page, 60, 60, seed=2)
    k, v = rows((1, 1, n, d), 1, torch.float32, 0.05), rows((1, 1, n, d), 2, torch.float32)
    q = rows((1, 4, Sq, d), 4, torch.float32, 0.1)
    q[..., 0] = 8.0
    k[0, 0, :, 0] = torch.arange(n) // 150 * 20.0  # scores rise by 20 every 150 keys
    v *= torch.exp2(torch.tensor([0, 9, -12, 3, 14, -6, 1])[torch.arange(n) // 48 % 7])[:, None]
    v[0, 0, 200:210] *= 2.0 ** 25  # large, but outweighed
    pkg.cache_append(c, k.cuda(), v.cuda(), dev(t), dev([0]))
    for causal in (True, False):
        check_attention(q.to(torch.bfloat16), c, t, [n], [Sq], causal, scale=1.0 / 8)
        # falling scores: the first reference is the last
        check_attention(-q.to(torch.bfloat16), c, t, [n], [Sq], causal, scale=1.0 / 8)


def test_marked_pages_with_many_rows():
    """As above in the 128-row kernel: a page's NaN reaches the rows that see it only."""
    page, d, n = 32, 128, 300
    c = new_cache(12, 1, page, d, "e4m3")
    t = tables([n], page, 12, 12, seed=5)
    k, v = rows((1, 1, n, d), 1, torch.float32), rows((1, 1, n, d), 2, torch.float32)
    v[0, 0, 290, 3] = math.nan  # page 9
    pkg.cache_append(c, k.cuda(), v.cuda(), dev(t), dev([0]))
    q = rows((1, 2, 40, d), 3, torch.bfloat16).cuda()  # positions 260 .. 299; page 9 begins at 288
    o, lse = pkg.attention_cache(q, c, dev(t), dev([n]))
    assert status() == pkg.ATTN_OK
    assert torch.isfinite(o[:, :, :28]).all() and torch.isnan(o[:, :, 28:]).all()
    assert torch.isfinite(lse).all()
    bad = t.copy()
    bad[0, 2] = 99
    pkg.attention_cache(q, c, dev(bad), dev([n]))
    assert status() == pkg.ATTN_ERR_TABLE


def _random_case(rng):
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    Hkv, G = rng.choice([1, 2, 3, 5]), rng.choice([1, 2, 3, 4, 7, 8, 9, 16, 33])
    Sq = rng.choice([1, 1, 2, 3, 5, 9, 17, 40])
    B = rng.randint(1, 4)
    most = rng.choice([3, 40, 150, 600])
    lens = [rng.choice([0, 1, rng.randint(1, most), rng.randint(1, most)]) for _ in range(B)]
    counts = [rng.randint(0, Sq) if rng.random() < 0.4 else Sq for _ in range(B)]
    return d, page, Hkv, G, Sq, lens, counts


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "L%s_q%d_H%dx%d_d%d_p%d" % (c[0], c[2], *c[3:]))
def test_a_wide_table_gives_the_same_results(case):
    """A table with room for long sequences has the work cut into ranges that cross the
    sequences; a narrow one gives each unit a CTA where units are few."""
    lens, counts, Sq, H, Hkv, d, page = case
    for fmt, dtype, out in (("e4m3", torch.bfloat16, None), ("int8", torch.float32, None),
                            ("e4m3", torch.float16, torch.float32)):
        c, t = filled(lens, Hkv, page, d, fmt, seed=len(lens) + d, width=8192 // page)
        q = rows((len(lens), H, Sq, d), 78, dtype)
        check_attention(q, c, t, lens, counts, True, out_dtype=out)
        pages = np.full((len(lens), Hkv, Sq, 80), -1)  # every page of the sequence, from the last
        for b, n in enumerate(lens):
            held = min(-(-n // page), 80)
            pages[b, ..., :held] = np.arange(held)[::-1]
        check_attention(q, c, t, lens, counts, False, out_dtype=out, pages=pages)


@pytest.mark.parametrize("d,fmt", [(64, "e4m3"), (64, "int8"), (128, "e4m3"), (128, "int8")])
def test_many_rows_of_many_sequences(d, fmt):
    """The 128-row kernel with more units than SMs, of uneven lengths, some without a token or a
    query: ranges hold several units, and units several ranges."""
    import random
    rng = random.Random(d)
    lens = [rng.choice([0, 1, 16, 127, 128, 129, rng.randint(1, 400)]) for _ in range(60)] + [1500]
    counts = [rng.choice([34, 34, 0, 1, 20]) for _ in lens]
    c, t = filled(lens, 3, 32, d, fmt, seed=d)
    q = rows((len(lens), 3, 34, d), 5, torch.bfloat16)
    for causal in (True, False):
        check_attention(q, c, t, lens, counts, causal)


def test_offsets_past_32_bits():
    """One sequence of 2^25 + 100 tokens: codes and rows lie past 2^32 bytes and elements.  All
    tokens but the last 200 are zeros, whose part of the softmax is a count."""
    page, d, n, m = 128, 128, 2 ** 25 + 100, 200
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    width = -(-n // page)
    c = new_cache(width + 1, 1, page, d, "e4m3")
    t = torch.arange(width, dtype=torch.int32, device="cuda")[None].contiguous()
    t[0, 7], t[0, -2] = width, 7  # the last three pages: near the pool's end, its start, its end
    t[0, -3], t[0, -1] = width - 1, width - 3
    last = [width - 1, 7, width - 3]
    k, v = rows((1, 1, m, d), 1, torch.bfloat16, 0.5), rows((1, 1, m, d), 2, torch.bfloat16)
    pkg.cache_append(c, k.cuda(), v.cuda(), t, dev([n - m]))
    assert status() == pkg.ATTN_OK

    def part(at):  # these pages in a pool of their own
        return pkg.KVCache(*(x[at] for x in (c.k, c.v, c.k_scale, c.v_scale, c.k_bounds)))

    small, own = part(last), [[0, 1, 2]]
    held = n - (width - 3) * page  # tokens in the last three pages
    want = ref.read(ref.snapshot(small), own, [held], held)
    assert abs(want[0]).max() > 1
    for dtype in (torch.bfloat16, torch.float16):
        for g, w in zip(pkg.cache_read(c, t, dev([n]), n, dtype=dtype), want):
            same(f64(g[:, :, n - held:]), f64(torch.from_numpy(w).to(dtype)))
            assert not g[:, :, : n - held: 4099].any()
    mixed = False
    for Sq, dtype in ((1, torch.float32), (1, torch.bfloat16), (5, torch.bfloat16), (40, torch.float16)):
        q = rows((1, 2, Sq, d), Sq, dtype)
        o, lse = pkg.attention_cache(q.cuda(), c, t, dev([n]), scale=0.12)
        assert status() == pkg.ATTN_OK
        o_, lse_, a, vmax = ref.attention(f64(q), ref.snapshot(small), own, [held], [Sq], True, 0.12)
        all_ = np.logaddexp(lse_, math.log(n - held))  # the other tokens' scores are 0
        share = np.exp(lse_ - all_)[..., None]
        mixed = mixed or np.any((share > 0.05) & (share < 0.95))
        # as check_attention, and two joins by lse, rounded by 2^-20 (below 32) each
        tol = 2 * 20 * 2.0 ** -23 * a + 2 * (2.0 ** -21 + 2.0 ** -12) + 2.0 ** -18 + 2.0 ** -17
        assert np.all(np.abs(f64(o) - o_ * share) <= tol * vmax + HALF[o.dtype] * np.abs(o_ * share) * 1.01)
        assert np.all(np.abs(f64(lse) - all_) <= tol)
    assert mixed
    near = t[:, -40:].contiguous()
    tokens, small = 39 * page + n % page, part(near[0].long())
    q, own = rows((1, 2, 1, d), 9, torch.float32), [list(range(40))]
    pages = pkg.cache_select(q.cuda(), c, near, dev([tokens]), 3).cpu().numpy()
    assert np.array_equal(pages, ref.select(f64(q), ref.snapshot(small), own, [tokens], [1], 3, True))
    o, _ = pkg.attention_cache(q.cuda(), c, near, dev([tokens]), pages=dev(pages))
    o_ = check_attention(q, small, np.array(own), [tokens], [1], True, pages=pages)[0]
    assert torch.equal(o, o_)
    assert status() == pkg.ATTN_OK


def test_scratch_grows_with_the_calls():
    """The workspace that a cache keeps serves small calls, larger ones and small ones again."""
    c, t = filled([900, 40], 2, 32, 64, "int8", seed=6)
    for Sq in (1, 40, 1, 6, 150, 1):
        q = rows((2, 4, Sq, 64), Sq, torch.float16)
        check_attention(q, c, t, [900, 40], [Sq, min(Sq, 3)], True)


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes(seed):
    """Head groups, lengths, counts, page sizes and types at random, all pages and selected ones."""
    import random
    rng = random.Random(seed)
    d, page, Hkv, G, Sq, lens, counts = _random_case(rng)
    while G * Hkv * Sq * sum(lens) > 400000:  # the reference is a loop over rows
        d, page, Hkv, G, Sq, lens, counts = _random_case(rng)
    fmt, causal = rng.choice(["e4m3", "int8"]), rng.random() < 0.6
    dtype = rng.choice([torch.bfloat16, torch.float16, torch.float32])
    out = torch.float32 if rng.random() < 0.3 else None
    c, t = filled(lens, Hkv, page, d, fmt, seed=seed, width=-(-max(max(lens), 1) // page) + rng.randint(0, 40))
    q = rows((len(lens), G * Hkv, Sq, d), seed + 9, dtype)
    check_attention(q, c, t, lens, counts, causal, out_dtype=out)
    n = rng.randint(1, 6)
    pages = pkg.cache_select(q.cuda(), c, dev(t), dev(lens), n, counts=dev(counts), causal=causal).cpu().numpy()
    assert np.array_equal(pages, ref.select(f64(q), ref.snapshot(c), t, lens, counts, n, causal))
    check_attention(q, c, t, lens, counts, causal, out_dtype=out, pages=pages)


def test_every_key_of_a_large_split_call_counts():
    """Long sequences: many partial states per row.  q = 0 gives equal weights, so o is the mean
    of v and lse the logarithm of the number of keys."""
    lens, page, d = [20000, 4097, 1], 64, 128
    c, t = filled(lens, 2, page, d, "int8", seed=8, dtype=torch.float16)
    q = torch.zeros((3, 4, 1, d), dtype=torch.float32, device="cuda")
    o, lse = pkg.attention_cache(q, c, dev(t), dev(lens))
    _, v = pkg.cache_read(c, dev(t), dev(lens), max(lens), dtype=torch.float32)
    assert status() == pkg.ATTN_OK
    for b, n in enumerate(lens):
        mean = v[b, :, :n].double().mean(1).repeat_interleave(2, 0)
        bound = (2.0 ** -20 + 2.0 ** -18) * v.abs().max().item()
        assert (o[b, :, 0].double() - mean).abs().max().item() <= bound
        assert (lse[b].double() - math.log(n)).abs().max().item() <= 2.0 ** -20 + 2.0 ** -22 * math.log(n)


def test_results_follow_neither_the_page_order_nor_the_batch():
    """The same sequence alone and in a batch, with other pages: the same within the sums' order,
    and bit for bit when repeated."""
    lens, page, d = [777, 1500, 20], 32, 128
    c, t = filled(lens, 2, page, d, "e4m3", seed=2, width=60)
    q = rows((3, 8, 2, d), 6, torch.float32).cuda()
    o, lse = pkg.attention_cache(q, c, dev(t), dev(lens))
    again, _ = pkg.attention_cache(q, c, dev(t), dev(lens))
    assert torch.equal(o, again)
    alone, _ = pkg.attention_cache(q[:1].contiguous(), c, dev(t[:1]), dev(lens[:1]))
    assert (alone - o[:1]).abs().max().item() <= 1e-4
    assert status() == pkg.ATTN_OK


def test_outputs_beside_the_call_stay():
    """Guard rows around o and lse, and the workspace's own bytes are enough."""
    lens, d = [100, 65], 64
    c, t = filled(lens, 2, 16, d, "e4m3")
    q = rows((2, 4, 3, d), 1, torch.bfloat16).cuda()
    st, need = pkg.attn_fwd_cache_workspace_size(2, 4, 2, 3, d, pkg.ATTN_BF16)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    o = torch.full((4, 4, 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 4, 3), 7.0, device="cuda")
    tt, ll = dev(t), dev(lens)
    st = pkg.attn_fwd_cache(c.c, q.data_ptr(), o[1].data_ptr(), lse[1].data_ptr(), tt.data_ptr(), t.shape[1],
                            ll.data_ptr(), None, None, 0, 2, 4, 3, 1, 0.0, pkg.ATTN_BF16, ws.data_ptr(), need, None)
    assert st == pkg.ATTN_OK and status() == pkg.ATTN_OK
    assert (o[0] == 7).all() and (o[3] == 7).all() and (lse[0] == 7).all() and (lse[3] == 7).all()
    assert (ws[need:] == 0xA5).all()
    w, wl = pkg.attention_cache(q, c, tt, ll)
    assert torch.equal(o[1:3], w) and torch.equal(lse[1:3], wl)


# ------------------------------------------------------------------ selection
SELECT = [
    # lens, counts, Sq, H, H_kv, d, page, n
    ([1], [1], 1, 1, 1, 64, 16, 1),
    ([400, 90], [1, 1], 1, 4, 2, 64, 16, 6),
    ([1000, 0, 130], [2, 2, 1], 2, 6, 2, 128, 32, 4),
    ([3000], [3], 3, 8, 1, 128, 16, 40),
    ([520, 260], [1, 1], 1, 16, 8, 64, 64, 3),
    ([700], [1], 1, 2, 2, 64, 16, 1),
    ([900, 300], [1, 1], 1, 40, 2, 128, 32, 7),           # 20 heads on one: three blocks of eight
    ([5000], [1], 1, 2, 1, 64, 16, 9),                    # pages for a whole cluster
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", SELECT, ids=lambda c: "L%s_q%d_n%d" % (c[0], c[2], c[7]))
def test_selection_and_attention_over_it(case, causal, dtype, fmt):
    lens, counts, Sq, H, Hkv, d, page, n = case
    c, t = filled(lens, Hkv, page, d, fmt, seed=n)
    q = rows((len(lens), H, Sq, d), 31, dtype)
    pages = pkg.cache_select(q.cuda(), c, dev(t), dev(lens), n, counts=dev(counts), causal=causal)
    assert status() == pkg.ATTN_OK
    want = ref.select(f64(q), ref.snapshot(c), t, lens, counts, n, causal)
    assert np.array_equal(pages.cpu().numpy(), want)
    check_attention(q, c, t, lens, counts, causal, pages=want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_selection_of_equal_and_almost_equal_scores(fmt):
    """Equal scores go to the lowest page; scores that fp32 sums cannot tell apart are told apart."""
    page, d, n_pages = 16, 64, 60
    c = new_cache(n_pages, 1, page, d, fmt)
    t = np.arange(n_pages)[None, ::-1].copy()
    k = torch.zeros((1, 1, n_pages * page, d))
    k[..., 0] = 64.0
    k[..., 1] = 2.0 ** -1 if fmt == "e4m3" else 1.0
    for p in (7, 20, 33):  # a shade more: the smallest step of a small channel
        k[0, 0, p * page, 1] *= 1.125 if fmt == "e4m3" else 2.0
    pkg.cache_append(c, k.cuda(), k.cuda(), dev(t), dev([0]))
    q = torch.zeros((1, 1, 1, d))
    q[..., 0] = 1024.0
    q[..., 1] = 2.0 ** -12  # 64 * 1024 + 2^-13 * (1 or 1.125): below fp32's step
    lens = [n_pages * page]
    for n in (1, 2, 3, 5, 30, 60, 64):
        pages = pkg.cache_select(q.cuda(), c, dev(t), dev(lens), n)
        want = ref.select(f64(q), ref.snapshot(c), t, lens, [1], n, True)
        assert np.array_equal(pages.cpu().numpy(), want)
    zero = pkg.cache_select(torch.zeros_like(q).cuda(), c, dev(t), dev(lens), 5).cpu().tolist()
    assert zero[0][0][0] == [0, 1, 2, 3, 59]
    assert status() == pkg.ATTN_OK


def test_selection_with_values_that_are_not_finite():
    page, d = 16, 64
    c, t = filled([160], 1, page, d, "e4m3", seed=1, dtype=torch.float32)
    x = rows((1, 1, 16, d), 2, torch.float32)
    x[0, 0, 3, 3] = math.nan
    pkg.cache_append(c, x.cuda(), x.cuda(), dev(t), dev([64]))  # page 4 is marked
    q = rows((1, 2, 1, d), 3, torch.float32)
    pages = pkg.cache_select(q.cuda(), c, dev(t), dev([160]), 3)
    assert np.array_equal(pages.cpu().numpy(), ref.select(f64(q), ref.snapshot(c), t, [160], [1], 3, True))
    assert 4 in pages.cpu().flatten().tolist()
    q[0, 0, 0, 0] = math.nan  # every page scores NaN: the lowest ones
    pages = pkg.cache_select(q.cuda(), c, dev(t), dev([160]), 3)
    assert pages.cpu().flatten().tolist() == [0, 1, 9]
    assert status() == pkg.ATTN_OK


def test_a_page_list_may_skip_repeat_and_name_unseen_pages():
    lens, page, d = [100], 16, 64
    c, t = filled(lens, 2, page, d, "int8", seed=4, width=9)
    q = rows((1, 4, 2, d), 3, torch.float32)
    listed = np.array([[[[0, -1, 3, 8], [-1, -1, -1, -1]], [[6, 2, -1, 2], [5, 4, 3, 2]]]])
    check_attention(q, c, t, lens, [2], True, pages=listed)


# ------------------------------------------------------------------ bad numbers from the device
def test_numbers_out_of_range_are_skipped_and_reported():
    lens, page, d = [64, 64], 16, 64
    c, t = filled(lens, 1, page, d, "e4m3", seed=6)
    q = rows((2, 1, 1, d), 1, torch.float32).cuda()
    x = rows((2, 1, 3, d), 2, torch.float32).cuda()
    good, _ = pkg.attention_cache(q, c, dev(t), dev(lens))
    assert status() == pkg.ATTN_OK
    for bad in (-1, -2 ** 31, c.n_pages, 2 ** 31 - 1):
        tt = t.copy()
        tt[0, 2] = bad
        o, _ = pkg.attention_cache(q, c, dev(tt), dev(lens))  # as if page 2 were not listed
        assert status() == pkg.ATTN_ERR_TABLE
        assert status() == pkg.ATTN_OK  # reported once
        w, _, _, _ = ref.attention(f64(q), ref.snapshot(c), t, lens, [1, 1], True,
                                   pages=np.array([[[[0, 1, 3, -1]]], [[[0, 1, 2, 3]]]]))
        assert np.abs(f64(o) - w).max() <= 1e-4 and torch.equal(o[1], good[1])
        k, _ = pkg.cache_read(c, dev(tt), dev(lens), 64)
        assert status() == pkg.ATTN_ERR_TABLE
        assert (k[0, :, 32:48] == 0).all() and not (k[0, :, 48:] == 0).all()
        pkg.cache_select(q, c, dev(tt), dev(lens), 2)
        assert status() == pkg.ATTN_ERR_TABLE
        before = ref.snapshot(c)
        pkg.cache_append(c, x, x, dev(tt), dev([40, 70]))  # a bad page, and rows past the table
        assert status() == pkg.ATTN_ERR_TABLE
        check_pool(c, before)
    for bad_lens in ([65, 64], [-1, 64], [2 ** 31 - 1, 64]):
        o, _ = pkg.attention_cache(q, c, dev(t), dev(bad_lens))
        assert status() == pkg.ATTN_ERR_TABLE
        assert torch.equal(o[1], good[1])
        assert bool((o[0] == 0).all()) == (bad_lens[0] < 0)
        pkg.cache_read(c, dev(t), dev(bad_lens), 64)
        assert status() == pkg.ATTN_ERR_TABLE
        pkg.cache_select(q, c, dev(t), dev(bad_lens), 2)
        assert status() == pkg.ATTN_ERR_TABLE
    before = ref.snapshot(c)
    for pos, counts in (([-1, -1], [1, 1]), ([0, 0], [4, -1])):
        pkg.cache_append(c, x, x, dev(t), dev(pos), dev(counts))
        assert status() == pkg.ATTN_ERR_TABLE
    check_pool(c, before)
    pkg.attention_cache(q, c, dev(t), dev(lens), counts=dev([2, 1]))
    assert status() == pkg.ATTN_ERR_TABLE
    listed = np.array([[[[0, 4]]], [[[1, -2]]]])
    pkg.attention_cache(q, c, dev(t), dev(lens), pages=dev(listed))
    assert status() == pkg.ATTN_ERR_TABLE


# ------------------------------------------------------------------ as it is used
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_serving_loop_with_prompt_chunk_drafts_and_single_tokens(fmt):
    """Two sequences: prompts, a chunk, three draft tokens of which one is taken back, then single
    tokens over selected pages; each step against the definition."""
    H, Hkv, d, page, width = 4, 2, 64, 16, 12
    c = new_cache(30, Hkv, page, d, fmt, junk=True)
    t = tables([width * page] * 2, page, width, 30, seed=3)
    pool = ref.snapshot(c)
    held, seed = [0, 0], 0
    for counts, Sq, keep in (([40, 23], 40, 0), ([0, 30], 30, 0), ([3, 3], 3, 1), ([1, 1], 1, 0), ([1, 1], 1, 0)):
        seed += 1
        k, v = rows((2, Hkv, Sq, d), seed, torch.bfloat16, seed), rows((2, Hkv, Sq, d), 50 + seed, torch.bfloat16)
        q = rows((2, H, Sq, d), 90 + seed, torch.bfloat16)
        pkg.cache_append(c, k.cuda(), v.cuda(), dev(t), dev(held), dev(counts))
        ref.append(pool, f64(k), f64(v), t, held, counts, fmt)
        lens = [a + b for a, b in zip(held, counts)]
        check_pool(c, pool)
        pages = None
        if Sq == 1:
            pages = pkg.cache_select(q.cuda(), c, dev(t), dev(lens), 3).cpu().numpy()
            assert np.array_equal(pages, ref.select(f64(q), pool, t, lens, counts, 3, True))
        check_attention(q, c, t, lens, counts, True, pages=pages)
        held = [n - keep for n in lens]  # a draft token that was not accepted is written over


def test_read_feeds_the_16_bit_attention():
    """cache_read's output through attention() and the cache's own attention agree."""
    n, H, d = 384, 2, 128
    c, t = filled([n], H, 64, d, "e4m3", seed=5)
    q = rows((1, H, n, d), 4, torch.bfloat16).cuda()
    k, v = pkg.cache_read(c, dev(t), dev([n]), n)
    a, la = pkg.attention(q, k, v, causal=True, out_dtype=torch.float32)
    b, lb = pkg.attention_cache(q, c, dev(t), dev([n]), out_dtype=torch.float32)
    assert status() == pkg.ATTN_OK
    # attention() rounds its weights to bf16 (2^-8 of each, numerator and sum); e4m3 codes are exact in bf16
    assert (a - b).abs().max().item() <= 2 * 2.0 ** -8 * v.float().abs().max().item()
    assert (la - lb).abs().max().item() <= 1e-4 * max(1.0, lb.abs().max().item())


def test_a_captured_step_follows_the_lengths_on_the_device():
    """One captured graph of append, select and attention, replayed as the sequences grow."""
    H, Hkv, d, page, width = 4, 2, 64, 16, 8
    caches = [new_cache(20, Hkv, page, d, "e4m3") for _ in range(2)]
    t = dev(tables([width * page] * 2, page, width, 20, seed=3))
    pos, lens = dev([30, 5]), dev([31, 6])
    x = rows((2, Hkv, 40, d), 1, torch.bfloat16).cuda()
    for c in caches:
        pkg.cache_append(c, x, x, t, dev([0, 0]), dev([30, 5]))
    k = torch.zeros((2, Hkv, 1, d), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, H, 1, d), dtype=torch.bfloat16, device="cuda")

    def step(c):
        pkg.cache_append(c, k, k, t, pos)
        pages = pkg.cache_select(q, c, t, lens, 2)
        return pages, *pkg.attention_cache(q, c, t, lens, pages=pages), *pkg.attention_cache(q, c, t, lens)

    spare = new_cache(20, Hkv, page, d, "e4m3")
    step(spare)  # set-up happens outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step(caches[0])
    for i in range(12):
        k.copy_(rows(k.shape, 10 + i, torch.bfloat16, 1 + i))
        q.copy_(rows(q.shape, 60 + i, torch.bfloat16))
        g.replay()
        direct = step(caches[1])
        for a, b in zip(captured, direct):
            assert torch.equal(a, b)
        pos += 1
        lens += 1
    assert status() == pkg.ATTN_OK
    check_pool(caches[0], ref.snapshot(caches[1]))


def test_calls_of_two_threads_on_one_stream():
    """Two threads decode with one cache on the default stream: a call's second kernel may come
    behind the other thread's first."""
    import threading
    lens, d = [2500, 900], 64
    c, t = filled(lens, 2, 32, d, "int8", seed=3)
    tt, ll = dev(t), dev(lens)
    qs = [[rows((2, 4, 1, d), 10 * k + i, torch.bfloat16).cuda() for i in range(20)] for k in range(2)]
    want = [[pkg.attention_cache(q, c, tt, ll) for q in x] for x in qs]
    torch.cuda.synchronize()
    got = [[], []]

    def work(k):
        for q in qs[k]:
            got[k].append(pkg.attention_cache(q, c, tt, ll))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    for k in range(2):
        for (a, la), (b, lb) in zip(want[k], got[k]):
            assert torch.equal(a, b) and torch.equal(la, lb)
    assert status() == pkg.ATTN_OK


def test_two_graphs_replayed_at_once():
    """Each captured call has a workspace of its own."""
    lens, d = [3000, 700], 64
    c, t = filled(lens, 2, 32, d, "e4m3", seed=3)
    tt, ll = dev(t), dev(lens)
    qs = [rows((2, 4, n, d), n, torch.bfloat16).cuda() for n in (1, 40)]
    want = [pkg.attention_cache(q, c, tt, ll) for q in qs]
    torch.cuda.synchronize()
    graphs, got = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(pkg.attention_cache(q, c, tt, ll))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (a, la), (b, lb) in zip(want, got):
        assert torch.equal(a, b) and torch.equal(la, lb)
    assert status() == pkg.ATTN_OK


@pytest.mark.parametrize("Sq", [1, 40])
def test_calls_on_two_streams_at_once(Sq):
    lens, d = [3000, 1200], 128
    c, t = filled(lens, 4, 64, d, "e4m3", seed=1)
    tt, ll = dev(t), dev(lens)
    qs = [rows((2, 8, Sq, d), i, torch.bfloat16).cuda() for i in range(8)]
    want = [pkg.attention_cache(q, c, tt, ll) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i, q in enumerate(qs):
        with torch.cuda.stream(streams[i % 2]):
            got.append(pkg.attention_cache(q, c, tt, ll))
    torch.cuda.synchronize()
    for (a, la), (b, lb) in zip(want, got):
        assert torch.equal(a, b) and torch.equal(la, lb)
    # the stream argument, with a workspace of the caller's
    st, need = pkg.attn_fwd_cache_workspace_size(2, 8, 4, Sq, d, pkg.ATTN_BF16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    o, _ = pkg.attention_cache(qs[0], c, tt, ll, workspace=ws, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(o, want[0][0]) and status() == pkg.ATTN_OK


def test_results_on_a_named_stream_share_no_memory_with_the_current_one():
    """Memory freed on the current stream may still be written by what is queued there; a call
    that names another stream gets its tensors from that one's."""
    lens, d = [900, 300], 64
    c, t = filled(lens, 2, 32, d, "e4m3", seed=1)
    tt, ll = dev(t), dev(lens)
    q = rows((2, 4, 1, d), 3, torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    calls = [lambda s: pkg.attention_cache(q, c, tt, ll, stream=s), lambda s: pkg.cache_read(c, tt, ll, 300, stream=s),
             lambda s: (pkg.cache_select(q, c, tt, ll, 3, stream=s),)]
    for f in calls:
        want = [x.clone() for x in f(None)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        late = [torch.empty_like(x).fill_(7) for x in want for _ in range(4)]
        del late  # freed, and written once the wait is over
        got = f(side)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    assert status() == pkg.ATTN_OK


def test_wrappers_refuse_before_launching():
    c, t = filled([40], 2, 16, 64, "e4m3")
    t, lens = dev(t), dev([40])
    x = torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    calls = [
        lambda: pkg.cache_append(c, x.cpu(), x.cpu(), t, lens),
        lambda: pkg.cache_append(c, x, x.float(), t, lens),
        lambda: pkg.cache_append(c, x.double(), x.double(), t, lens),
        lambda: pkg.cache_append(c, x[:, :1], x[:, :1], t, lens),
        lambda: pkg.cache_append(c, x, x, t.long(), lens),
        lambda: pkg.cache_append(c, x, x, t[0], lens),
        lambda: pkg.cache_append(c, x, x, t, lens, counts=dev([1, 1])),
        lambda: pkg.cache_append(c, x, x, t, lens.cpu()),
        lambda: pkg.cache_append(c, x.expand(1, 2, 5, 64), x.expand(1, 2, 5, 64), t, lens),
        lambda: pkg.cache_read(c, t, lens, 40, dtype=torch.float64),
        lambda: pkg.cache_read(c, t, lens, 40, out=(x, x)),
        lambda: pkg.cache_read(c, t, lens, -1),
        lambda: pkg.cache_read(c, lens[0], lens, 40),
        lambda: pkg.attention_cache(q, c, t, lens, pages=lens[0]),
        lambda: pkg.cache_select(q, c, t, lens, 0),
        lambda: pkg.cache_select(q[:, :3], c, t, lens, 1),
        lambda: pkg.attention_cache(q[..., :32], c, t, lens),
        lambda: pkg.attention_cache(q, c, t, lens, out_dtype=torch.float16),
        lambda: pkg.attention_cache(q, c, t, lens, pages=dev([[[[0]]]])),
        lambda: pkg.attention_cache(q, c, t, lens, pages=torch.zeros((1, 2, 1, 1), dtype=torch.int64, device="cuda")),
        lambda: pkg.attention_cache(q, c, t, lens, workspace=torch.zeros(1 << 24, dtype=torch.uint8)),
    ]
    for i, f in enumerate(calls):
        with pytest.raises(ValueError):
            f()
            raise AssertionError("call %d was not refused" % i)
    with pytest.raises(pkg.AttnError):
        pkg.attention_cache(q, c, t, lens, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert status() == pkg.ATTN_OK


# ------------------------------------------------------------------ the bounds-checking build
def test_checked_build_finds_no_index_out_of_bounds():
    ensure_built()
    lib = pkg.load_checked_library()
    s = torch.cuda.current_stream().cuda_stream
    for fmt in ("e4m3", "int8"):
        for lens, counts, Sq, H, Hkv, d, page in ATTEND:
            B = len(lens)
            c, t = filled(lens, Hkv, page, d, fmt, seed=1)
            tt, ll, cc = dev(t), dev(lens), dev(counts)
            q = rows((B, H, Sq, d), 2, torch.bfloat16).cuda()
            x = torch.empty((B, Hkv, 45, d), dtype=torch.bfloat16, device="cuda")
            y = torch.empty_like(x)
            assert lib.attn_cache_read(c.c, tt.data_ptr(), t.shape[1], ll.data_ptr(), x.data_ptr(), y.data_ptr(),
                                       B, 45, pkg.ATTN_BF16, s) == pkg.ATTN_OK
            o, lse = torch.empty_like(q), torch.empty((B, H, Sq), device="cuda")
            pages = torch.empty((B, Hkv, Sq, 2), dtype=torch.int32, device="cuda")
            ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
            assert lib.attn_cache_select(c.c, q.data_ptr(), tt.data_ptr(), t.shape[1], ll.data_ptr(), cc.data_ptr(),
                                         pages.data_ptr(), 2, B, H, Sq, 1, pkg.ATTN_BF16, ws.data_ptr(), ws.numel(),
                                         s) == pkg.ATTN_OK
            for p, n in ((None, 0), (pages.data_ptr(), 2)):
                assert lib.attn_fwd_cache(c.c, q.data_ptr(), o.data_ptr(), lse.data_ptr(), tt.data_ptr(), t.shape[1],
                                          ll.data_ptr(), cc.data_ptr(), p, n, B, H, Sq, 1, 0.0, pkg.ATTN_BF16,
                                          ws.data_ptr(), ws.numel(), s) == pkg.ATTN_OK
            z = torch.zeros((B, Hkv, 9, d), dtype=torch.bfloat16, device="cuda")
            pos = dev([0] * B)
            n = dev([min(9, m) for m in lens])
            assert lib.attn_cache_append(c.c, z.data_ptr(), z.data_ptr(), tt.data_ptr(), t.shape[1], pos.data_ptr(),
                                         n.data_ptr(), B, 9, pkg.ATTN_BF16, s) == pkg.ATTN_OK
            assert lib.attn_check_status(None) == pkg.ATTN_OK
            w = pkg.attention_cache(q, *filled(lens, Hkv, page, d, fmt, seed=1)[:1], tt, ll, counts=cc,
                                    pages=pages)[0]
            assert torch.equal(w, o)
