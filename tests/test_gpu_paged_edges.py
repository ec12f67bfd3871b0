"""Edges of the paged 8-bit KV cache and its attention: batches of hundreds of
sequences, far pages, shared pages, NaN codes behind a mask, other streams, a
workspace that many calls use, rows past the batch.  Same oracle and bound as
the main tests."""
import numpy as np
import pytest
import torch

from gpu_util import to_dev
from oracle import paged
from test_gpu_paged import D, E4M3, INT8, attend, bound, device_cache, i32, page_table, random_cache, same_cache
from ternary_weight_decode_b200 import tern

pytestmark = pytest.mark.gpu


def close(out, q, start, ctx, pages, ref, kind, window=0, sinks=0):
    """out (the rows of a call) against the oracle."""
    T = int(start[-1])
    want = paged.attention(q[:T], start, ctx, pages, ref, kind, window, sinks)
    k_ref, v_ref, _ = paged.values(np.concatenate([[0], np.cumsum(np.maximum(ctx, 0))]), ctx, pages, ref, kind)
    err = np.abs(out[:T].cpu().numpy() - want)
    tol = bound(q, k_ref, v_ref, D ** -0.5, max(ctx))
    assert np.all(err <= tol), (float(err.max()), tol)


def mid_cache(rng, kind, Hkv, page, n_pages):
    """A random cache whose e4m3 exponents lie in the middle of the range."""
    ref = random_cache(rng, kind, Hkv, page, n_pages)
    if kind == E4M3:
        for x in ("k_codes", "v_codes"):
            ref[x] = (ref[x] & 0x8F) | (((ref[x] >> 4 & 3) + 3) << 4).astype(np.uint8)
        ref = {k: (a * 4 if "scales" in k else a) for k, a in ref.items()}
    return ref


# ---------------------------------------------------------------- masks
@pytest.mark.parametrize("window,sinks", [(1, 1), (17, 20), (64, 3), (5000, 4)])
@pytest.mark.parametrize("n,ctx,page", [([1, 1], [90, 513], 16), ([7, 2], [140, 260], 64), ([150], [280], 48)])
def test_window_and_sinks_e4m3(n, ctx, page, window, sinks):
    attend(np.random.default_rng(window + sinks), n, ctx, page, E4M3, 10, 2, window, sinks)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0, 1e-20])
def test_scales_e4m3(scale):
    attend(np.random.default_rng(9), [1, 6], [70, 150], 16, E4M3, 10, 2, scale=scale)
    attend(np.random.default_rng(9), [80], [150], 16, E4M3, 10, 2, scale=scale)


@pytest.mark.parametrize("n,ctx,Hq,Hkv,page", [([1], [20011], 40, 8, 64), ([5, 16], [9001, 4100], 10, 2, 32),
                                               ([300], [5000], 4, 1, 128)])
def test_long_contexts_e4m3(n, ctx, Hq, Hkv, page):
    attend(np.random.default_rng(12), n, ctx, page, E4M3, Hq, Hkv)


@pytest.mark.parametrize("n", [4, 12, 90])
@pytest.mark.parametrize("window", [0, 7])
def test_nan_codes_reach_only_the_rows_that_see_them(n, window):
    """A NaN code in a token's key or value makes the rows that see the token
    NaN, and every other row is what it is without it."""
    rng = np.random.default_rng(n)
    Hq, Hkv, page, L, at = 6, 2, 32, n + 150, n + 150 - n // 2  # the token lies in the middle of the rows
    pages, n_pages = page_table(rng, [L], page)
    ref = mid_cache(rng, E4M3, Hkv, page, n_pages)
    q = rng.standard_normal((n, Hq, D)).astype(np.float32)
    want = paged.attention(q, [0, n], [L], pages, ref, E4M3, window, 0)
    k_ref, v_ref, _ = paged.values([0, L], [L], pages, ref, E4M3)
    tol = bound(q, k_ref, v_ref, D ** -0.5, L)
    batch = tern.PagedBatch(i32([0, n]), i32([L]), i32(pages), n, n, L)
    ws = tern.attention_paged_workspace(Hq, device_cache(ref, E4M3))

    first = at - (L - n)                       # rows first .. last - 1 see the token
    last = n if window == 0 else min(n, first + window)
    others = np.ones((n, Hq), bool)
    others[first:last, :3] = False             # query heads 0..2 read KV head 0
    for part, code in (("k_codes", 0x7F), ("v_codes", 0xFF)):
        bad = {k: a.copy() for k, a in ref.items()}
        bad[part][pages[0, at // page], 0, at % page, 5] = code
        out = torch.full((n, Hq, D), -2.0, device="cuda")
        tern.tern_attention_paged(to_dev(q), batch, device_cache(bad, E4M3), out, ws, window=window)
        out = out.cpu().numpy()
        assert np.all(np.abs(out - want)[others] <= tol)
        assert np.all(np.isnan(out[~others][:, 5]))


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_queries_that_are_not_finite(n, value, kind):
    """Their rows are NaN (0 where nothing is seen), the others what they are."""
    rng = np.random.default_rng(n)
    Hq, Hkv, page, ctx = 6, 2, 32, [n + 300, n - 1 if n > 1 else 40]
    pages, n_pages = page_table(rng, ctx, page)
    ref = mid_cache(rng, kind, Hkv, page, n_pages)
    start = np.array([0, n, 2 * n])
    q = rng.standard_normal((2 * n, Hq, D)).astype(np.float32)
    want = paged.attention(q, start, ctx, pages, ref, kind)
    k_ref, v_ref, _ = paged.values(np.array([0, ctx[0], sum(ctx)]), ctx, pages, ref, kind)
    tol = bound(q, k_ref, v_ref, D ** -0.5, max(ctx))
    bad = np.zeros((2 * n, Hq), bool)
    bad[n - 1, 1] = bad[n, 4] = bad[2 * n - 1, 0] = True   # row n sees nothing when n > 1
    q[bad, 77] = value
    dev = device_cache(ref, kind)
    out = torch.full((2 * n, Hq, D), -2.0, device="cuda")
    tern.tern_attention_paged(to_dev(q), tern.PagedBatch(i32(start), i32(ctx), i32(pages), 2 * n, n, max(ctx)), dev, out,
                              tern.attention_paged_workspace(Hq, dev))
    out = out.cpu().numpy()
    assert np.all(np.abs(out - want)[~bad] <= tol)
    if n > 1:
        assert np.all(out[n] == 0)
        bad[n] = False
    assert np.all(np.isnan(out[bad]))


# ---------------------------------------------------------------- many sequences
@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("B", [256, 257, 300, 1000])
def test_many_sequences(B, kind):
    """More sequences than a CTA has threads to count them, some without rows."""
    rng = np.random.default_rng(B)
    n = [int(x) for x in rng.choice([0, 1, 1, 1, 3], B)]
    ctx = [int(a + x) for a, x in zip(n, rng.integers(0, 90, B))]
    attend(rng, n, ctx, 16, kind, 6, 2)


def test_most_sequences():
    n = [1] * 4096
    attend(np.random.default_rng(1), n, [1 + i % 37 for i in range(4096)], 16, INT8, 2, 1)


@pytest.mark.parametrize("kind", [INT8, E4M3])
def test_append_of_many_sequences(kind):
    rng = np.random.default_rng(300)
    B, Hq, Hkv, page = 300, 3, 1, 16
    n = [int(x) for x in rng.choice([0, 1, 2, 20], B)]
    ctx = [int(a + x) for a, x in zip(n, rng.integers(0, 50, B))]
    T = sum(n)
    pages, n_pages = page_table(rng, ctx, page)
    start = np.concatenate([[0], np.cumsum(n)])
    ref = random_cache(rng, kind, Hkv, page, n_pages)
    dev = device_cache(ref, kind)
    table = paged.rope_table(10000.0, D, 80)
    q, k, v = (rng.standard_normal((T, h, D)).astype(np.float32) for h in (Hq, Hkv, Hkv))
    pos = rng.integers(0, 80, (1, T)).astype(np.int32)
    q_out = torch.empty(T, Hq, D, device="cuda")
    batch = tern.PagedBatch(i32(start), i32(ctx), i32(pages), T, max(n), max(ctx))
    tern.tern_kv_append_paged(to_dev(q), to_dev(k), to_dev(v), to_dev(pos), tern.RopePlan(to_dev(table)), batch, dev, q_out)
    q_ref, _ = paged.append(q, k, v, pos, table, start, ctx, pages, ref, kind)
    np.testing.assert_array_equal(q_out.cpu().numpy(), q_ref)
    same_cache(dev, ref)


def test_rows_past_the_batch_buffers():
    """row_start may name more rows than T: the rows from T on are neither read
    nor written, those before keep their places in their sequences."""
    rng = np.random.default_rng(31)
    Hq, Hkv, page, n, ctx = 6, 2, 16, [3, 9], [40, 70]
    pages, n_pages = page_table(rng, ctx, page)
    ref = mid_cache(rng, INT8, Hkv, page, n_pages)
    start = np.array([0, 3, 12])
    q = rng.standard_normal((12, Hq, D)).astype(np.float32)
    want = paged.attention(q, start, ctx, pages, ref, INT8)
    k_ref, v_ref, _ = paged.values(np.array([0, 40, 110]), ctx, pages, ref, INT8)
    tol = bound(q, k_ref, v_ref, D ** -0.5, 70)
    dev = device_cache(ref, INT8)
    ws = tern.attention_paged_workspace(Hq, dev)
    for T in (1, 3, 4, 11):
        buf, out = to_dev(q.copy()), torch.full((12, Hq, D), -2.0, device="cuda")
        buf[T:] = float("nan")
        tern.tern_attention_paged(buf[:T], tern.PagedBatch(i32(start), i32(ctx), i32(pages), T, 9, 70), dev, out[:T], ws)
        assert np.all(np.abs(out[:T].cpu().numpy() - want[:T]) <= tol)
        assert torch.all(out[T:] == -2.0)


# ---------------------------------------------------------------- pages
@pytest.mark.parametrize("kind", [INT8, E4M3])
def test_far_pages(kind):
    """Pages more than 2^32 bytes into the code arrays."""
    rng = np.random.default_rng(40)
    Hq, Hkv, page, ctx, n = 6, 2, 64, [200, 131], [3, 1]
    n_pages = (1 << 32) // (Hkv * page * D) + 40
    small_pages, n_small = page_table(rng, ctx, page)
    ref = mid_cache(rng, kind, Hkv, page, n_small)
    place = n_pages - 1 - 3 * np.arange(n_small)   # where each of the small cache's pages lies in the large one
    pages = np.where(small_pages >= 0, place[np.maximum(small_pages, 0)], -1).astype(np.int32)
    dev = tern.PagedCache.empty(kind, Hkv, D, page, n_pages)
    for x in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(dev, x).view(n_pages, -1)[torch.as_tensor(place).cuda()] = to_dev(ref[x]).view(n_small, -1)
    start = np.array([0, 3, 4])
    table = paged.rope_table(10000.0, D, 256)
    q, k, v = (rng.standard_normal((4, h, D)).astype(np.float32) for h in (Hq, Hkv, Hkv))
    pos = np.array([[197, 198, 199, 130]], np.int32)
    batch = tern.PagedBatch(i32(start), i32(ctx), i32(pages), 4, 3, 200)
    q_out, out = torch.empty(4, Hq, D, device="cuda"), torch.empty(4, Hq, D, device="cuda")
    tern.tern_kv_append_paged(to_dev(q), to_dev(k), to_dev(v), to_dev(pos), tern.RopePlan(to_dev(table)), batch, dev, q_out)
    q_ref, _ = paged.append(q, k, v, pos, table, start, ctx, small_pages, ref, kind)
    for x in ("k_codes", "k_scales", "v_codes", "v_scales"):
        got = getattr(dev, x).view(n_pages, -1)[torch.as_tensor(place).cuda()].cpu().numpy()
        np.testing.assert_array_equal(got, ref[x].reshape(n_small, -1))
    tern.tern_attention_paged(q_out, batch, dev, out, tern.attention_paged_workspace(Hq, dev))
    close(out, q_ref, start, ctx, small_pages, ref, kind)
    k_out, v_out = torch.empty(4, Hkv, D, device="cuda"), torch.empty(4, Hkv, D, device="cuda")
    tern.tern_kv_read_paged(batch, dev, k_out, v_out)
    k_ref, v_ref, _ = paged.values(start, ctx, small_pages, ref, kind)
    np.testing.assert_array_equal(k_out.cpu().numpy(), k_ref)
    np.testing.assert_array_equal(v_out.cpu().numpy(), v_ref)


def test_sequences_that_share_pages():
    """A common prefix held once, and one page named twice by a sequence."""
    rng = np.random.default_rng(41)
    Hq, Hkv, page, ctx, n = 10, 2, 32, [100, 90, 64], [1, 5, 1]
    pages = np.array([[3, 1, 0, 4], [3, 1, 2, -1], [1, 1, -1, -1]], np.int32)
    ref = mid_cache(rng, INT8, Hkv, page, 5)
    dev = device_cache(ref, INT8)
    start = np.array([0, 1, 6, 7])
    q = rng.standard_normal((7, Hq, D)).astype(np.float32)
    out = torch.empty(7, Hq, D, device="cuda")
    tern.tern_attention_paged(to_dev(q), tern.PagedBatch(i32(start), i32(ctx), i32(pages), 7, 5, 100), dev, out,
                              tern.attention_paged_workspace(Hq, dev))
    close(out, q, start, ctx, pages, ref, INT8)


def test_descriptors_follow_their_tensors():
    """A tensor whose memory or size changes in place, or a field replaced, is seen by the next call."""
    rng = np.random.default_rng(42)
    Hq, Hkv, page = 4, 2, 16
    pages = np.array([[0, 1, 2], [3, 4, 5]], np.int32)
    ref = mid_cache(rng, INT8, Hkv, page, 6)
    dev = device_cache(ref, INT8)
    ws = tern.attention_paged_workspace(Hq, dev)
    q = rng.standard_normal((2, Hq, D)).astype(np.float32)
    batch = tern.PagedBatch(i32([0, 1, 2]), i32([20, 30]), i32(pages), 2, 1, 48)

    def check(n, ctx):
        out = torch.full((n, Hq, D), -2.0, device="cuda")
        tern.tern_attention_paged(to_dev(q[:n]), batch, dev, out, ws)
        close(out, q[:n], np.arange(n + 1), ctx, pages, ref, INT8)
    check(2, [20, 30])
    batch.ctx.set_(i32([48, 3]))
    check(2, [48, 3])
    other = mid_cache(rng, INT8, Hkv, page, 6)
    for x in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(dev, x).data = to_dev(other[x])
    ref = other
    check(2, [48, 3])
    batch.ctx.resize_(1)
    batch.row_start.resize_(2)
    batch.pages.resize_(1, 3)
    batch.T = 1
    check(1, [48])

    table = paged.rope_table(10000.0, D, 40)
    plan = tern.RopePlan(to_dev(table), [10, 54])
    pos = np.array([[3, 9], [30, 1]], np.int32)
    for sections in ([10, 54], [60, 4]):
        plan.sections[:] = sections
        y = torch.empty(2, Hq, D, device="cuda")
        tern.tern_rope(plan, to_dev(pos), to_dev(q), y)
        np.testing.assert_array_equal(y.cpu().numpy(), paged.rope(q, pos, table, sections)[0])


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("n,ctx,Hq,Hkv,page,window", [([1, 3], [700, 5], 71, 1, 4096, 0), ([2], [260], 128, 1, 112, 33),
                                                      ([37], [4200], 3, 3, 4096, 0), ([1], [1030], 64, 64, 16, 0)])
def test_large_groups_and_pages(n, ctx, Hq, Hkv, page, window, kind):
    """Many query heads on one KV head, many KV heads, the largest page, and one no power of two divides."""
    attend(np.random.default_rng(Hq), n, ctx, page, kind, Hq, Hkv, window=window, sinks=2)


# ---------------------------------------------------------------- streams, graphs, workspaces
class Call:
    def __init__(self, seed, n, ctx, kind, Hq, Hkv, page=32, window=0):
        rng = np.random.default_rng(seed)
        self.n, self.ctx, self.kind, self.window = n, ctx, kind, window
        self.pages, n_pages = page_table(rng, ctx, page)
        self.ref = mid_cache(rng, kind, Hkv, page, n_pages)
        self.dev = device_cache(self.ref, kind)
        self.start = np.concatenate([[0], np.cumsum(n)])
        self.q = rng.standard_normal((sum(n), Hq, D)).astype(np.float32)
        self.dq, self.out = to_dev(self.q), torch.full((sum(n), Hq, D), -2.0, device="cuda")
        self.batch = tern.PagedBatch(i32(self.start), i32(ctx), i32(self.pages), sum(n), max(n), max(ctx))

    def run(self, ws):
        tern.tern_attention_paged(self.dq, self.batch, self.dev, self.out, ws, window=self.window)

    def check(self):
        close(self.out, self.q, self.start, self.ctx, self.pages, self.ref, self.kind, self.window)
        self.out.fill_(-2.0)


def some_calls():
    return [Call(1, [1, 1], [5000, 77], INT8, 10, 2), Call(2, [40], [900], E4M3, 4, 4), Call(3, [1], [9000], E4M3, 8, 1),
            Call(4, [70, 2], [400, 2100], INT8, 6, 1, window=100), Call(5, [1] * 20, [150] * 20, INT8, 40, 8)]


def test_one_workspace_for_many_calls():
    """Calls of other sizes, heads and kinds, one after another, eager and in one graph."""
    calls = some_calls()
    ws = tern.attention_paged_workspace(10, calls[0].dev)
    for c in calls + calls[::-1]:
        c.run(ws)
    for c in calls:
        c.check()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        for c in calls:
            c.run(ws)
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other, stream=side):  # a second graph on the same workspace, replayed in turn
        for c in calls[::-1]:
            c.run(ws)
    for g in (graph, other, graph):
        g.replay()
        torch.cuda.synchronize()
        for c in calls:
            c.check()


def test_two_streams_with_a_workspace_each():
    calls = some_calls()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [tern.attention_paged_workspace(10, calls[0].dev) for _ in streams]
    twins = some_calls()
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ws, mine in zip(streams, spaces, (calls, twins[::-1])):
            with torch.cuda.stream(s):
                for c in mine:
                    c.run(ws)
    torch.cuda.synchronize()
    for a, b in zip(calls, twins):
        assert torch.equal(a.out, b.out)
        a.check()


def test_the_same_batch_twice_gives_the_same_bits_beside_other_work():
    c, noise = Call(6, [1, 1, 7], [3000, 4500, 60], INT8, 10, 2), Call(7, [50], [800], E4M3, 10, 2)
    ws, ws2, side = tern.attention_paged_workspace(10, c.dev), tern.attention_paged_workspace(10, c.dev), torch.cuda.Stream()
    c.run(ws)
    first = c.out.clone()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(side):
            noise.run(ws2)
        c.run(ws)
        assert torch.equal(c.out, first)
    torch.cuda.synchronize()
    noise.check()
