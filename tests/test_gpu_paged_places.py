"""Attention over page tables with missing entries in front of the cache's
first page: the place behind a missing block's is that of block 0, which must
not be taken for its continuation.  (The copies' division itself is checked on
the host, tests/test_paged_copies.py.)  And values too large for any scale."""
import numpy as np
import pytest
import torch

from gpu_util import to_dev
from oracle import paged
from test_gpu_paged import D, E4M3, INT8, i32
from test_gpu_paged_edges import close, device_cache, mid_cache
from ternary_weight_decode_b200 import tern

pytestmark = pytest.mark.gpu

TABLES = [  # page size, pages of each sequence, contexts
    (16, [[-1, 0]], [32]), (16, [[-1, 0, 7, 9, 3, 4, 5]], [100]), (16, [[-1, 0, 1, 2, 3, 4, 5, 6, 7]], [140]),
    (16, [[5, 6, 7, -1, 0, 1, 2, 3, 4], [8, -1, -1, 0, 1, -1, 0, 1, 2]], [139, 144]),
    (48, [[-1, 0, 1], [2, -1, 0]], [140, 129]), (112, [[-1, 0, 1], [-1, 0, -1]], [300, 200]),
    (16, [[9, 3, -1, 0, 1, 2, 99, 0, 5, -1, 0, 1, 2, 3, 4, 6, 7]], [270])]


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("rows,Hq,Hkv", [(1, 4, 1), (1, 20, 2), (5, 6, 1), (21, 4, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 20), (33, 0)])
@pytest.mark.parametrize("page,pages,ctx", TABLES)
def test_first_page_behind_a_missing_one(page, pages, ctx, window, sinks, rows, Hq, Hkv, kind):
    rng = np.random.default_rng(page + sum(ctx) + rows)
    pages = np.array(pages, np.int32)
    B = len(ctx)
    ref = mid_cache(rng, kind, Hkv, page, 10)
    dev = device_cache(ref, kind)
    start = np.arange(B + 1) * rows
    q = rng.standard_normal((B * rows, Hq, D)).astype(np.float32)
    out = torch.full((B * rows, Hq, D), -2.0, device="cuda")
    tern.tern_attention_paged(to_dev(q), tern.PagedBatch(i32(start), i32(ctx), i32(pages), B * rows, rows, max(ctx)), dev,
                              out, tern.attention_paged_workspace(Hq, dev), window=window, sinks=sinks)
    close(out, q, start, ctx, pages, ref, kind, window, sinks)
    assert tern.tern_device_error() == 0


@pytest.mark.parametrize("kind", [INT8, E4M3])
def test_values_beyond_the_largest_scale_saturate(kind):
    """The scale stops at 2^120; what lies above the largest code of it is the largest code, of either
    sign, when it is written and when earlier tokens are rescaled."""
    rng = np.random.default_rng(5)
    Hkv, page, L = 2, 16, 20
    table = paged.rope_table(10000.0, D, 40)
    ref = mid_cache(rng, kind, Hkv, page, 2)
    dev = device_cache(ref, kind)
    pages = np.array([[1, 0]], np.int32)
    x = rng.standard_normal((L, Hkv, D))
    x[:, 0] *= 1e38
    x[3, 1, 5], x[4, 1, 6], x[17, 1, 7], x[17, 0, 8] = -3e38, 3e38, -3.4e38, 3.4e38
    x = np.clip(x, -3.4e38, 3.4e38).astype(np.float32)
    for t0, t1 in ((0, 2), (2, 5), (5, 20)):
        n = t1 - t0
        # position 0: the rotation leaves the values as they are
        args = x[t0:t1], x[t0:t1], x[t0:t1], np.zeros((1, n), np.int32)
        out = torch.empty(n, Hkv, D, device="cuda")
        tern.tern_kv_append_paged(*map(to_dev, args), tern.RopePlan(to_dev(table)),
                                  tern.PagedBatch(i32([0, n]), i32([t1]), i32(pages), n, n, t1), dev, out)
        paged.append(*args, table, [0, n], [t1], pages, ref, kind)
        for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
            np.testing.assert_array_equal(getattr(dev, name).cpu().numpy(), ref[name], err_msg=name)
