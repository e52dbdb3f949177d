"""The paged 8-bit cache at the edges of what a call may be given: sequences that take no part."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import online_softmax_forward_gb300 as pkg
from test_gpu_cache import check_pool, dev, f64, new_cache, rows, status

pytestmark = pytest.mark.gpu


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
