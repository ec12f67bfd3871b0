"""Attention over page tables with missing entries in front of the cache's
first page: the place behind a missing block's is that of block 0, which must
not be taken for its continuation.  (The copies' division itself is checked on
the host, tests/test_paged_copies.py.)"""
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
