"""The paged 8-bit cache where a wrong number hides behind a large one: rows bounded by what they
themselves weigh, page scales that span the type's range, sequences that take no part in a call,
selections that many pages tie in.

Attention is compared row by row and channel by channel.  With w_j the softmax weights of a row:

  s     a score is off by e_s = 20 * 2^-23 * a, a the largest sum_c |q_c k_c| * scale (as in
        test_gpu_cache.py), so a weight by 2 e_s of itself (numerator and sum);
  p     exp2 and the products with the page scale: 2^-21 of a weight; rounded to fp16 for 16-bit
        outputs: 2^-11 of it, half a step;
  sums  n / 16 products of 16 keys and a few joins and rescalings one behind the other, 2^-23 of
        what the sum has reached: (n / 16 + 16) * 2^-23 each for o and for the weights' sum;
  low   a weight that leaves fp16's normal numbers is rounded to steps of 2^-24, half a step off;
        one that the row weighs most, by weight times page scale, stands at no less than 2^5 (the
        128-row kernel's reference; 2^11 in the other): 2^-30 * |code| * max_j w_j v_scale_j a key;
  out   half a step of the output type (and of fp16's subnormals, 2^-25).
"""
import math

import numpy as np
import pytest
import torch

import cache_ref as ref
import online_softmax_forward_gb300 as pkg
import test_gpu_cache as cache_tests
from gpu_util import ensure_built
from test_gpu_cache import HALF, check_pool, dev, f64, new_cache, rows, status, tables

pytestmark = pytest.mark.gpu


def check_rows(q, c, t, n, Sq, causal=True, scale=None, out_dtype=None):
    """attention_cache of one sequence of n tokens, H_kv = 1, each row and channel within its own bound."""
    o, lse = pkg.attention_cache(q.cuda(), c, dev(t), dev([n]), causal=causal, scale=scale, out_dtype=out_dtype)
    assert status() == pkg.ATTN_OK
    pool, page, d = ref.snapshot(c), c.page, c.d
    k, v = (x[0, 0] for x in ref.read(pool, t, [n], n))
    ids = [t[0][j // page] for j in range(n)]
    vs = pool["v_scale"][ids, 0]
    code = np.abs(np.stack([pool["v"][p, 0, j % page] for j, p in enumerate(ids)]))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    got, glse = f64(o), f64(lse)
    ep = 2.0 ** -21 + (2.0 ** -11 if o.dtype != torch.float32 else 0.0)
    sums = 2 * (n / 16 + 16) * 2.0 ** -23
    tight = 0.0
    for h in range(q.shape[1]):
        for i in range(Sq):
            m = ref.visible(n, Sq, i, causal)
            x = f64(q[0, h, i])
            s = k[:m] @ x * scale
            es = 20 * 2.0 ** -23 * (np.abs(k[:m]) @ np.abs(x) * scale).max()
            w = np.exp(s - s.max())
            o_, lse_ = w @ v[:m] / w.sum(), s.max() + math.log(w.sum())
            own = w @ np.abs(v[:m]) / w.sum()
            low = 2.0 ** -30 * (w * vs[:m]).max() * code[:m].sum(0) / w.sum()
            bound = (2 * es + ep + sums) * own + low + HALF[o.dtype] * np.abs(o_) * 1.01
            bound += 2.0 ** -25 if o.dtype == torch.float16 else 2.0 ** -149
            err = np.abs(got[0, h, i] - o_)
            worst = (err / bound).argmax()
            assert np.all(err <= bound), "head %d query %d channel %d: %r, not %r, bound %.3e" % (
                h, i, worst, got[0, h, i, worst], o_[worst], bound[worst])
            assert abs(glse[0, h, i] - lse_) <= es + 2.0 ** -20 + 2.0 ** -22 * abs(lse_)
            tight = max(tight, np.median(bound / np.maximum(own, 1e-300)))
    assert tight < 2.0 ** -3  # the bound says something about o
    return o


def one_sequence(k, v, page, fmt, seed=0):
    """(cache, table) of one sequence of one kv head; k and v [n, d]."""
    n, d = k.shape
    pages = -(-n // page)
    c = new_cache(pages + 2, 1, page, d, fmt, junk=True)
    t = tables([n], page, pages, pages + 2, seed=seed)
    pkg.cache_append(c, k[None, None].cuda(), v[None, None].cuda(), dev(t), dev([0]))
    assert status() == pkg.ATTN_OK
    return c, t


ROWS = [(1, torch.bfloat16), (4, torch.float16), (7, torch.bfloat16), (40, torch.bfloat16),  # 8 to 128 rows
        (3, torch.float32)]


# ------------------------------------------------------------------ sequences that take no part
@pytest.mark.parametrize("page", [16, 64])
def test_append_of_no_rows_touches_no_page(page):
    """A sequence with a count of 0 in the middle of a page: its table row may name pages that are
    another's by now, or none at all."""
    d = 64
    c = new_cache(6, 2, page, d, "e4m3")
    x = rows((2, 2, 9, d), 1, torch.bfloat16)
    pool = ref.snapshot(c)
    ref.append(pool, f64(x[1:]), f64(-x[1:]), [[3, 4]], [0], [9], "e4m3")
    for other in (-1, 99):
        t = np.array([[other, other], [3, 4]])
        pkg.cache_append(c, x.cuda(), (-x).cuda(), dev(t), dev([7, 0]), dev([0, 9]))
        assert status() == pkg.ATTN_OK
        check_pool(c, pool)


def test_append_of_no_rows_beside_the_pages_new_owner():
    """The row of a sequence that left still names a page which another starts in the same call."""
    d, page = 128, 16
    for r in range(20):
        c = new_cache(70, 2, page, d, "int8")
        c.k_scale.fill_(8.0)
        c.v_scale.fill_(16.0)
        B = 64
        x = rows((2 * B, 2, 3, d), r, torch.float16)
        t = np.concatenate([np.arange(B), np.arange(B)])[:, None]
        pos = [5] * B + [0] * B
        counts = [0] * B + [3] * B
        pool = ref.snapshot(c)
        ref.append(pool, f64(x), f64(x), t, pos, counts, "int8")
        pkg.cache_append(c, x.cuda(), x.cuda(), dev(t), dev(pos), dev(counts))
        assert status() == pkg.ATTN_OK
        check_pool(c, pool)


# ------------------------------------------------------------------ page scales far apart
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Sq,dtype", ROWS)
def test_a_large_page_of_no_weight_behind_pages_of_zeros(Sq, dtype, fmt):
    """The first keys that a row weighs have zero values, then come pages of huge ones whose
    weights underflow, then ordinary ones."""
    n, d = 700, 64
    k, v = rows((n, d), 1, torch.float32, 0.05), rows((n, d), 2, torch.float32)
    k[:, 0] = 0.0
    v[:448] = 0.0
    k[448:512, 0] = -200.0
    v[448:512] *= 1e25
    c, t = one_sequence(k, v, 16, fmt)
    q = rows((1, 4, Sq, d), 4, torch.float32, 0.1)
    q[..., 0] = 8.0
    check_rows(q.to(dtype), c, t, n, Sq, scale=1.0 / 8)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Sq,dtype", ROWS)
@pytest.mark.parametrize("wide", [False, True])
def test_large_values_that_scores_leave_behind_for_zeros(wide, Sq, dtype, fmt):
    """Huge values first, then a score so much higher that nothing of them is left, on pages of
    zeros, then ordinary values."""
    n, d = 900, 64
    k, v = rows((n, d), 1, torch.float32, 0.05), rows((n, d), 2, torch.float32)
    k[:, 0] = 200.0
    head = 64 if not wide else 32
    for at in range(0, 512, 2 * head):
        k[at: at + head, 0] = 0.0
        v[at: at + head] *= 1e30
        v[at + head: at + 2 * head] = 0.0
    c, t = one_sequence(k, v, 16, fmt)
    q = rows((1, 4, Sq, d), 4, torch.float32, 0.1)
    q[..., 0] = 8.0
    check_rows(q.to(dtype), c, t, n, Sq, scale=1.0 / 8)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Sq,dtype", ROWS)
@pytest.mark.parametrize("at,far,low", [(0, 34, -19.0), (48, 34, -19.0), (304, 36, -20.0), (300, 20, -8.0)])
def test_an_outweighed_page_costs_the_others_no_bits(at, far, low, Sq, dtype, fmt):
    """One page whose scale is 2^far of the others' and whose keys weigh e^low of theirs, large in
    channel 0 only: the other channels are sums of ordinary values."""
    n, d = 600, 64
    k, v = rows((n, d), 1, torch.float32, 0.05), rows((n, d), 2, torch.float32)
    k[:, 0] = 0.0
    k[at: at + 16, 0] = low
    v[at + 3, 0] = 2.0 ** far
    c, t = one_sequence(k, v, 16, fmt)
    q = rows((1, 4, Sq, d), 4, torch.float32, 0.1)
    q[..., 0] = 8.0
    check_rows(q.to(dtype), c, t, n, Sq, causal=False, scale=1.0 / 8)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Sq,dtype", ROWS)
@pytest.mark.parametrize("sign", [1, -1])
def test_moving_references_row_by_row(sign, Sq, dtype, fmt):
    """Scores that rise (or fall) by 20 every 150 keys while the pages' scales go up and down by
    many powers of two, among them outweighed pages of 2^25 more."""
    page, d, n = 16, 64, 900
    k, v = rows((n, d), 1, torch.float32, 0.05), rows((n, d), 2, torch.float32)
    k[:, 0] = torch.arange(n) // 150 * 20.0
    v *= torch.exp2(torch.tensor([0, 9, -12, 3, 14, -6, 1])[torch.arange(n) // 48 % 7])[:, None]
    v[200:210] *= 2.0 ** 25
    c, t = one_sequence(k, v, page, fmt, seed=2)
    q = rows((1, 4, Sq, d), 4, torch.float32, 0.1)
    q[..., 0] = 8.0
    for causal in (True, False):
        check_rows(sign * q.to(dtype), c, t, n, Sq, causal, scale=1.0 / 8)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Sq,dtype", ROWS)
@pytest.mark.parametrize("v_scale", [3.3e38, 2.0 ** 127, 2.0 ** 122, 2.0 ** -126])
def test_any_finite_scale_of_values(v_scale, Sq, dtype, fmt):
    """A pool filled by hand, codes of one and its neighbours under the largest and the smallest
    scale."""
    n, d, page = 200, 64, 16
    k = rows((n, d), 1, torch.float32, 0.3)
    v = torch.where(torch.arange(d) % 3 == 0, 1.0, 0.5 if fmt == "e4m3" else 0.0).expand(n, d).contiguous()
    c, t = one_sequence(k, v, page, fmt)
    c.v.copy_(torch.where(torch.arange(d) % 3 == 0, 1.0, 0.5 if fmt == "e4m3" else 0.0).to(c.v.dtype).cuda())
    c.v_scale.fill_(v_scale)
    q = rows((1, 4, Sq, d), 4, torch.float32).to(dtype)
    o, _ = pkg.attention_cache(q.cuda(), c, dev(t), dev([n]), out_dtype=torch.float32)
    assert status() == pkg.ATTN_OK
    want = f64(c.v[0, 0, 0].float()) * v_scale  # every key has the same value
    assert np.abs(f64(o) / v_scale - want / v_scale).max() <= 2.0 ** -18
    if dtype == torch.bfloat16:
        o, _ = pkg.attention_cache(q.cuda(), c, dev(t), dev([n]))
        assert np.abs(f64(o) / v_scale - want / v_scale).max() <= 2.0 ** -8 + 2.0 ** -10


# ------------------------------------------------------------------ selection
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,small", [(torch.float32, 1e-8), (torch.bfloat16, 1e-8), (torch.float32, 1e-4),
                                         (torch.float32, 1e-30)])
def test_selection_of_scores_below_normal_numbers(dtype, small, fmt):
    """Keys at the smallest scale under small queries: fp32 scores are subnormal or 0, the choice
    is that of their exact values."""
    n, d, page = 640, 64, 16
    k = rows((n, d), 1, torch.float32, 2.0 ** -124)
    c, t = one_sequence(k, k, page, fmt)
    assert (c.k_scale[torch.from_numpy(t[0]).cuda()] == 2.0 ** -126).all()
    q = (rows((1, 3, 2, d), 2, torch.float32) * small).to(dtype)
    for m in (2, 7, 20):
        pages = pkg.cache_select(q.cuda(), c, dev(t), dev([n]), m)
        assert status() == pkg.ATTN_OK
        want = ref.select(f64(q), ref.snapshot(c), t, [n], [2], m, True)
        assert np.array_equal(pages.cpu().numpy(), want)
        assert not np.array_equal(want[0, 0, 0, : m - 1], np.arange(m - 1))


def many_pages(pages, fmt="e4m3", page=16, seed=1, heads=1, d=64):
    """(cache, table, k, v): one sequence of so many pages of random rows."""
    n = pages * page
    c = new_cache(pages, heads, page, d, fmt)
    t = np.random.RandomState(seed).permutation(pages)[None]
    k = rows((1, heads, n, d), seed, torch.float32)
    return c, t, k


def check_selection(q, c, t, lens, ns):
    for n in ns:
        pages = pkg.cache_select(q.cuda(), c, dev(t), dev(lens), n)
        assert status() == pkg.ATTN_OK
        want = ref.select(f64(q), ref.snapshot(c), t, lens, [q.shape[2]], n, True)
        assert np.array_equal(pages.cpu().numpy(), want), n


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("pages", [200, 700, 2000])  # up to eight CTAs, few or many pages near the cut
@pytest.mark.parametrize("marked", [1, 5, 400])
def test_selection_among_marked_pages(marked, pages, fmt):
    """Pages that hold a value which is not finite score highest, the lowest of them first, and
    leave the others' order as it is."""
    c, t, k = many_pages(pages, fmt)
    at = np.random.RandomState(3).permutation(pages - 1)[: min(marked, pages // 2)]
    for i, p in enumerate(at):
        k[0, 0, 16 * p + i % 16, i % 64] = (math.nan, math.inf, -math.inf)[i % 3]
    pkg.cache_append(c, k.cuda(), k.cuda(), dev(t), dev([0]))
    for heads, dtype in ((2, torch.bfloat16), (9, torch.float32)):  # a block of eight heads, two
        check_selection(rows((1, heads, 2, 64), 2, dtype), c, t, [16 * pages],
                        (1, 2, len(at), len(at) + 1, len(at) + 2, len(at) + 40, pages - 1))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("pages", [300, 1500])
def test_selection_where_many_pages_tie(pages, fmt):
    """Equal scores, and scores that differ by less than fp32 tells, on more pages than are settled
    pair by pair; some far above and below."""
    c, t, k = many_pages(pages, fmt)
    k[:] = 0
    k[..., 0], k[..., 1] = 64.0, 0.5 if fmt == "e4m3" else 1.0
    rng = np.random.RandomState(5)
    for p in rng.permutation(pages)[: pages // 3]:
        k[0, 0, 16 * p, 1] *= 1.125 if fmt == "e4m3" else 2.0
    for i, p in enumerate(rng.permutation(pages)[:20]):
        k[0, 0, 16 * p: 16 * p + 16, 0] = 8.0 if i % 2 else 128.0
    pkg.cache_append(c, k.cuda(), k.cuda(), dev(t), dev([0]))
    q = torch.zeros((1, 1, 1, 64))
    q[..., 0], q[..., 1] = 1024.0, 2.0 ** -12
    ns = (1, 2, 5, 30, pages // 3, pages // 2, pages - 7, pages - 1, pages)
    check_selection(q, c, t, [16 * pages], ns)
    check_selection(-q, c, t, [16 * pages], ns)
    check_selection(q * 0, c, t, [16 * pages], ns)


def test_selection_of_a_query_that_is_not_finite():
    """Every page's score is NaN, infinite or, where codes are 0, as it may be."""
    pages = 600
    c, t, k = many_pages(pages)
    k[..., 3] = 0
    k[0, 0, 16 * 77: 16 * 78, 5] = 0
    k[0, 0, 16 * 99: 16 * 100] = 0
    pkg.cache_append(c, k.cuda(), k.cuda(), dev(t), dev([0]))
    for value in (math.nan, math.inf, -math.inf):
        for channel in (3, 5, 7):
            q = rows((1, 1, 1, 64), 2, torch.float32)
            q[0, 0, 0, channel] = value
            with np.errstate(invalid="ignore"):
                check_selection(q, c, t, [16 * pages], (2, 60, 300, 598))


def test_selection_of_marked_pages_and_zeros():
    """Scores of 0 wherever the page is not marked."""
    pages = 400
    c, t, k = many_pages(pages)
    k[:] = 0
    k[0, 0, 16 * 123] = math.nan
    pkg.cache_append(c, k.cuda(), k.cuda(), dev(t), dev([0]))
    for q in (rows((1, 1, 1, 64), 2, torch.float32), torch.zeros(1, 1, 1, 64)):
        check_selection(q, c, t, [16 * pages], (1, 2, 3, 50, 399))


def test_selection_takes_no_detour_for_marked_pages_or_ties():
    """4096 pages: neither a marked page nor equal scores may cost a multiple of milliseconds."""
    pages = 4096
    times = []
    for state in ("ordinary", "marked", "equal"):
        c, t, k = many_pages(pages)
        if state == "marked":
            k[0, 0, 16 * 1000 + 3, 5] = math.nan
        if state == "equal":
            k[:] = 1.0
        pkg.cache_append(c, k.cuda(), k.cuda(), dev(t), dev([0]))
        q, tt, ll = rows((1, 4, 1, 64), 2, torch.bfloat16).cuda(), dev(t), dev([16 * pages])
        best = math.inf
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            pkg.cache_select(q, c, tt, ll, 96)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    print("ordinary, marked, equal: %.3f %.3f %.3f ms" % tuple(times))
    assert status() == pkg.ATTN_OK
    assert times[1] < 4 * times[0] and times[2] < 2.0


# ------------------------------------------------------------------ memory and refusals
def test_workspaces_end_with_their_use():
    """Selecting for many queries among many pages leaves no workspace of its size behind, and a
    thread's workspaces end with the thread."""
    import threading
    pages = 2000
    c, t, k = many_pages(pages, heads=2)
    tt, ll = dev(t), dev([16 * pages])
    pkg.cache_append(c, k.cuda(), k.cuda(), tt, dev([0]))
    q = rows((1, 2, 2000, 64), 3, torch.bfloat16).cuda()
    one = q[:, :, :1].contiguous()
    pkg.attention_cache(one, c, tt, ll)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    del_me = pkg.cache_select(q, c, tt, ll, 3)
    del del_me
    assert torch.cuda.memory_allocated() - before < 8 << 20  # the call's own is 64 MB

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(3):
                pkg.attention_cache(one, c, tt, ll)
            torch.cuda.synchronize()

    before = torch.cuda.memory_allocated()
    for _ in range(8):
        x = threading.Thread(target=work)
        x.start()
        x.join()
    assert torch.cuda.memory_allocated() == before
    assert status() == pkg.ATTN_OK


def test_empty_pools_are_refused():
    for n, h in ((0, 2), (4, 0)):
        with pytest.raises(ValueError):
            pkg.KVCache.empty(n, h, 16, 64)


# ------------------------------------------------------------------ the bounds-checking build
@pytest.fixture
def checked(monkeypatch):
    """The wrappers on libattn_checked.so: status() then also reports an index out of bounds."""
    ensure_built()
    monkeypatch.setattr(pkg, "load_library", pkg.load_checked_library)


@pytest.mark.parametrize("case", cache_tests.ATTEND, ids=lambda c: "L%s_q%d_H%dx%d_d%d_p%d" % (c[0], c[2], *c[3:]))
def test_checked_wide_tables_and_lists(checked, case):
    cache_tests.test_a_wide_table_gives_the_same_results(case)


@pytest.mark.parametrize("d,fmt", [(64, "int8"), (128, "e4m3")])
def test_checked_shared_ranges(checked, d, fmt):
    cache_tests.test_many_rows_of_many_sequences(d, fmt)
    cache_tests.test_every_key_of_a_large_split_call_counts()


def test_checked_selection(checked):
    test_selection_among_marked_pages(5, 2000, "int8")
    test_selection_where_many_pages_tie(1500, "e4m3")
    for case in cache_tests.SELECT:
        cache_tests.test_selection_and_attention_over_it(case, True, torch.float32, "e4m3")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_checked_append_read_and_serving(checked, dtype):
    for case in cache_tests.APPEND:
        cache_tests.test_append_gives_the_definition(case, dtype, "int8")
    cache_tests.test_append_of_special_values("e4m3")
    for case in (([100, 7], 70, 3, 64, 64), ([129, 128, 1, 0], 140, 1, 128, 128)):
        cache_tests.test_read_gives_what_the_codes_stand_for(case, dtype, "e4m3")
    cache_tests.test_a_serving_loop_with_prompt_chunk_drafts_and_single_tokens("int8")
    cache_tests.test_numbers_out_of_range_are_skipped_and_reported()
