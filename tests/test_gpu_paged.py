"""GPU parity of the rotary embedding and the paged 8-bit KV cache.

Rotations, codes, scales and read-back values equal the numpy oracle bit for
bit (each step is one fp32 rounding, and the scales are powers of two).  The
attention is held to the 64-bit oracle within a bound counted from its
roundings (`bound` below)."""
import numpy as np
import pytest
import torch

from gpu_util import to_dev
from oracle import paged
from ternary_weight_decode_b200 import tern

pytestmark = pytest.mark.gpu
D = 128
INT8, E4M3 = tern.TERN_KV_INT8, tern.TERN_KV_E4M3


def i32(a):
    return to_dev(np.asarray(a, np.int32))


# ---------------------------------------------------------------- rotary embedding
def test_table_matches_fp64():
    plan = tern.RopePlan.build(1e6, 128, 70000, scale=0.25)
    ref = paged.rope_table(1e6, 128, 70000, 0.25)
    # both round the same fp64 value, each formed within an error far below an fp32 step: at most one step apart
    assert np.abs(plan.table.cpu().numpy() - ref).max() <= 2.0 ** -24


@pytest.mark.parametrize("T,H,d,rot,sections,inter,inverse,strided", [
    (1, 1, 8, 8, None, False, False, False), (1, 48, 128, 128, None, False, False, True),
    (37, 7, 128, 128, [16, 24, 24], False, False, True), (5, 3, 256, 64, [10, 22], False, True, False),
    (130, 2, 64, 64, [3, 9, 20], True, False, True), (33, 5, 80, 40, None, True, True, False),
    (3, 2, 512, 512, [0, 0, 256], False, False, False), (1000, 9, 128, 96, [1, 47], True, False, False)])
def test_rope_matches_oracle(T, H, d, rot, sections, inter, inverse, strided):
    rng = np.random.default_rng(T + H + d)
    axes = 1 if sections is None else len(sections)
    table = paged.rope_table(10000.0, rot, 777)
    pos = rng.integers(0, 777, (axes, T)).astype(np.int32)
    if T > 3:
        pos[axes - 1, 1], pos[0, 3] = 777, -1    # outside the table
    x = rng.standard_normal((T, H, d)).astype(np.float32)
    plan = tern.RopePlan(to_dev(table), sections, inter, inverse)
    wide = torch.full((T, H * d + 16), 7.0, device="cuda")
    xd = wide[:, 8:8 + H * d].view(T, H, d) if strided else torch.empty(T, H, d, device="cuda")
    xd.copy_(to_dev(x))
    y = torch.full((T, H, d), 3.0, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    tern.tern_rope(plan, to_dev(pos), xd, y, d_invalid=bad)
    ref, nbad = paged.rope(x, pos, table, sections, inter, inverse)
    np.testing.assert_array_equal(y.cpu().numpy(), ref)
    assert int(bad) == nbad
    tern.tern_rope(plan, to_dev(pos), xd, xd)    # in place
    np.testing.assert_array_equal(xd.cpu().numpy(), ref)
    if strided:
        assert torch.all(wide[:, :8] == 7.0) and torch.all(wide[:, 8 + H * d:] == 7.0)


def test_inverse_rotation_is_the_gradient():
    """d/dx of sum(w * rope(x)) is the rotation of w by the negative angles:
    against differences in 64 bits (exact for a linear map up to rounding)."""
    rng = np.random.default_rng(3)
    table = paged.rope_table(10000.0, 128, 50)
    pos = rng.integers(0, 50, (3, 4)).astype(np.int32)
    w = rng.standard_normal((4, 2, D)).astype(np.float32)
    g = torch.empty(4, 2, D, device="cuda")
    tern.tern_rope(tern.RopePlan(to_dev(table), [16, 24, 24], inverse=True), to_dev(pos), to_dev(w), g)
    tab = table.astype(np.float64)

    def f(x):
        y = np.empty_like(x)
        for t in range(4):
            c = np.concatenate([tab[pos[a, t], s] for a, s in enumerate((slice(0, 16), slice(16, 40), slice(40, 64)))])
            y[t, :, :64] = x[t, :, :64] * c[:, 0] - x[t, :, 64:] * c[:, 1]
            y[t, :, 64:] = x[t, :, 64:] * c[:, 0] + x[t, :, :64] * c[:, 1]
        return float((y * w).sum())

    x = rng.standard_normal((4, 2, D))
    got = g.cpu().numpy()
    for t, h, d in [(0, 0, 0), (1, 1, 63), (2, 0, 64), (3, 1, 127), (0, 1, 31)]:
        e = np.zeros_like(x)
        e[t, h, d] = 1.0
        # |w| up to 4, two products and a sum: three fp32 roundings of values up to 8
        assert abs((f(x + e) - f(x - e)) / 2 - got[t, h, d]) <= 3 * 8 * 2.0 ** -24 + 1e-12


# ---------------------------------------------------------------- cache
def random_cache(rng, kind, Hkv, page, n_pages):
    """A cache full of finite values that no call has written: garbage where tokens are still to come."""
    codes = [rng.integers(0, 256, (n_pages, Hkv, page, D), dtype=np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 127) == 127] = 5  # no NaN of e4m3, no -128 or -1 of int8 by accident of the mask
        c[c == 128] = 3
    scales = [np.exp2(rng.integers(-9, -5, (n_pages, Hkv, page // 16))).astype(np.float32) for _ in range(2)]
    return dict(k_codes=codes[0], v_codes=codes[1], k_scales=scales[0], v_scales=scales[1])


def device_cache(c, kind):
    n, Hkv, page, d = c["k_codes"].shape
    return tern.PagedCache(kind, Hkv, d, page, *(to_dev(c[x]) for x in ("k_codes", "k_scales", "v_codes", "v_scales")))


def same_cache(dev, ref):
    for x in ("k_codes", "k_scales", "v_codes", "v_scales"):
        np.testing.assert_array_equal(getattr(dev, x).cpu().numpy(), ref[x], err_msg=x)


def page_table(rng, ctx, page, ld_extra=1):
    per = [max(0, -(-c // page)) for c in ctx]
    ids = rng.permutation(sum(per) + 2)
    t = np.full((len(ctx), max(per) + ld_extra), -1, np.int32)
    at = 0
    for b, k in enumerate(per):
        t[b, :k] = ids[at:at + k]
        at += k
    return t, len(ids)


APPENDS = [  # rows and context of each sequence, page size, kind, Hq, Hkv
    ([1], [1], 16, INT8, 5, 1), ([1], [17], 16, E4M3, 40, 8), ([1], [32], 32, INT8, 40, 8),
    ([3, 0, 1, 16], [40, 9, 16, 48], 48, INT8, 8, 4), ([3, 0, 1, 16], [40, 9, 16, 48], 32, E4M3, 8, 4),
    ([70, 33], [70, 100], 64, INT8, 6, 3), ([200, 1, 15], [207, 1, 31], 128, E4M3, 4, 2),
    ([1] * 37, list(range(1, 38)), 16, INT8, 7, 1)]


@pytest.mark.parametrize("n,ctx,page,kind,Hq,Hkv", APPENDS)
@pytest.mark.parametrize("sections,inter", [(None, False), ([16, 24, 24], False), ([20, 44], True)])
def test_append_and_read_match_oracle(n, ctx, page, kind, Hq, Hkv, sections, inter):
    rng = np.random.default_rng(sum(n) + page)
    T, axes = sum(n), 1 if sections is None else len(sections)
    pad = 5  # rows behind the last sequence
    pages, n_pages = page_table(rng, ctx, page)
    start = np.concatenate([[0], np.cumsum(n)])
    ref = random_cache(rng, kind, Hkv, page, n_pages)
    dev = device_cache(ref, kind)
    table = paged.rope_table(10000.0, D, 300)
    plan = tern.RopePlan(to_dev(table), sections, inter)
    for scale in (0.01, 3.0, 0.5):  # the same rows again, larger and smaller: blocks whose scale grows, and stays
        qkv = (rng.standard_normal((T + pad, (Hq + 2 * Hkv) * D)) * scale).astype(np.float32)
        qkv[::3, Hq * D:Hq * D + 9] = 0.0
        pos = rng.integers(0, 300, (axes, T + pad)).astype(np.int32)
        if T > 4:
            pos[0, 2], pos[axes - 1, 4] = 300, -7
        q, k, v = (qkv[:, a * D:b * D].reshape(T + pad, b - a, D) for a, b in
                   ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        dq = to_dev(qkv)
        parts = [dq[:, a * D:b * D].view(T + pad, b - a, D) for a, b in
                 ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]
        q_out = torch.full((T + pad, Hq, D), -2.0, device="cuda")
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        batch = tern.PagedBatch(i32(start), i32(ctx), i32(pages), T + pad, max(max(n), 1), max(ctx))
        tern.tern_kv_append_paged(*parts, to_dev(pos), plan, batch, dev, q_out, d_invalid=bad)
        q_ref, nbad = paged.append(q, k, v, pos, table, start, ctx, pages, ref, kind, sections, inter)
        np.testing.assert_array_equal(q_out[:T].cpu().numpy(), q_ref[:T])
        assert torch.all(q_out[T:] == -2.0), "rows behind the last sequence stay as they were"
        same_cache(dev, ref)
        assert int(bad) == nbad
    k_out, v_out = (torch.full((T + pad, Hkv, D), -2.0, device="cuda") for _ in range(2))
    tern.tern_kv_read_paged(batch, dev, k_out, v_out)
    k_ref, v_ref, _ = paged.values(start, ctx, pages, ref, kind)
    np.testing.assert_array_equal(k_out[:T].cpu().numpy(), k_ref)
    np.testing.assert_array_equal(v_out[:T].cpu().numpy(), v_ref)
    assert torch.all(k_out[T:] == -2.0) and torch.all(v_out[T:] == -2.0)


def test_bad_pages_are_skipped_and_counted():
    rng = np.random.default_rng(11)
    page, Hkv, n, ctx = 32, 2, [40, 6, 4], [40, 100, 2]  # the last context is shorter than its rows
    pages = np.array([[1, -1], [9, 0], [2, 3]], np.int32)  # sequence 1: past its entries, sequence 0: none for 32..39
    start = np.concatenate([[0], np.cumsum(n)])
    T = sum(n)
    ref = random_cache(rng, INT8, Hkv, page, 5)
    dev = device_cache(ref, INT8)
    table = paged.rope_table(10000.0, D, 50)
    q, k, v = (rng.standard_normal((T, h, D)).astype(np.float32) for h in (4, 2, 2))
    pos = np.zeros((1, T), np.int32)
    batch = tern.PagedBatch(i32(start), i32(ctx), i32(pages), T, 40, 100)
    q_out, bad = torch.empty(T, 4, D, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    tern.tern_kv_append_paged(to_dev(q), to_dev(k), to_dev(v), to_dev(pos), tern.RopePlan(to_dev(table)), batch, dev,
                              q_out, d_invalid=bad)
    q_ref, nbad = paged.append(q, k, v, pos, table, start, ctx, pages, ref, INT8)
    assert nbad == 8 + 6 + 2 and int(bad) == nbad
    same_cache(dev, ref)
    np.testing.assert_array_equal(q_out.cpu().numpy(), q_ref)
    k_out, v_out = torch.empty(T, 2, D, device="cuda"), torch.empty(T, 2, D, device="cuda")
    bad.zero_()
    tern.tern_kv_read_paged(batch, dev, k_out, v_out, d_invalid=bad)
    k_ref, v_ref, nbad = paged.values(start, ctx, pages, ref, INT8)
    np.testing.assert_array_equal(k_out.cpu().numpy(), k_ref)
    np.testing.assert_array_equal(v_out.cpu().numpy(), v_ref)
    assert int(bad) == nbad


# ---------------------------------------------------------------- attention
def bound(q, vals_k, vals_v, scale, L):
    """Largest error of an output.  A score is a sum of 128 products in fp32
    (136 roundings of at most 2^-23 of A = scale sum |q_d k_d|, the splitting of
    q into two fp16 parts among them); its exponent in base 2 rounds |score| a
    few times more (8); a weight is off by twice that (numerator and
    denominator), and by 2^-20 for the exponential and its split.  The weighted
    sum adds at most 2^-23 a step over L / 16 + 64 steps."""
    g = q.shape[1] // vals_k.shape[1]
    A = abs(scale) * max(float(np.max(np.abs(q[:, h]) @ np.abs(vals_k[:, h // g]).T)) for h in range(q.shape[1]))
    return float(np.abs(vals_v).max()) * (2 * 144 * 2.0 ** -23 * A + 2.0 ** -20 + (L / 16 + 64) * 2.0 ** -23)


def attend(rng, n, ctx, page, kind, Hq, Hkv, window=0, sinks=0, scale=None, drop=None, max_rows=None, max_ctx=None,
           garbage_tail=True):
    pages, n_pages = page_table(rng, ctx, page)
    ref = random_cache(rng, kind, Hkv, page, n_pages)
    # e4m3: exponents in the middle of the range, so that no code dominates
    if kind == E4M3:
        for x in ("k_codes", "v_codes"):
            ref[x] = (ref[x] & 0x8F) | (((ref[x] >> 4 & 3) + 3) << 4).astype(np.uint8)
        ref = {k: (a * 4 if "scales" in k else a) for k, a in ref.items()}
    if drop is not None:
        drop(pages)
    start = np.concatenate([[0], np.cumsum(n)])
    T, pad = int(start[-1]), 3
    q = (rng.standard_normal((T + pad, Hq, D)) * 1.5).astype(np.float32)
    want = paged.attention(q[:T], start, ctx, pages, ref, kind, window, sinks, scale)
    k_ref, v_ref, _ = paged.values(np.concatenate([[0], np.cumsum(np.maximum(ctx, 0))]), ctx, pages, ref, kind)
    tol = bound(q, k_ref, v_ref, D ** -0.5 if scale is None else scale, max(ctx))
    if garbage_tail:  # what lies behind a context is never used, whatever it holds
        for b, c in enumerate(ctx):
            if c > 0 and c % page and 0 <= pages[b, c // page] < n_pages:
                pg, s = pages[b, c // page], c % page
                ref["k_codes"][pg, :, s:], ref["v_codes"][pg, :, s:] = 0x7F, 0xFF   # NaN in e4m3
                ref["k_scales"][pg, :, -(-s // 16):] = np.nan
                ref["v_scales"][pg, :, -(-s // 16):] = np.inf
    dev = device_cache(ref, kind)
    batch = tern.PagedBatch(i32(start), i32(ctx), i32(pages), T + pad, max_rows or max(max(n), 1),
                            max_ctx or max(max(ctx), 1))
    ws = tern.attention_paged_workspace(Hq, dev)
    ws[1024:] = float("nan")  # only the counters have to be zero
    outs = []
    for _ in range(2):
        out = torch.full((T + pad, Hq, D), -2.0, device="cuda")
        tern.tern_attention_paged(to_dev(q), batch, dev, out, ws, window=window, sinks=sinks, scale=scale)
        outs.append(out)
    got = outs[0].cpu().numpy()
    assert np.all(got[T:] == -2.0), "rows behind the last sequence stay as they were"
    assert torch.equal(outs[0], outs[1]), "the same inputs give the same bits"
    err = np.abs(got[:T] - want)
    assert np.all(err <= tol), (float(err.max()), tol, np.argwhere(~(err <= tol))[:4])
    assert not ws[:1024].view(torch.int32).any(), "the counters are zero again"
    assert tern.tern_device_error() == 0
    return got[:T]


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("Hq,Hkv", [(40, 8), (8, 8), (7, 1), (16, 2), (24, 2), (20, 1)])
@pytest.mark.parametrize("n,ctx,page", [([1], [1], 16), ([1], [16], 16), ([1], [17], 32), ([1], [333], 48),
                                        ([1, 1, 1], [5, 200, 64], 64), ([1, 0, 1], [31, 4, 129], 128)])
def test_attention_of_single_tokens(n, ctx, page, Hq, Hkv, kind):
    attend(np.random.default_rng(Hq + sum(ctx)), n, ctx, page, kind, Hq, Hkv)


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("Hq,Hkv", [(10, 2), (4, 4), (9, 1)])
@pytest.mark.parametrize("n,ctx,page", [([2], [2], 16), ([5], [300], 16), ([16, 3, 1], [40, 131, 77], 32),
                                        ([40], [40], 64), ([130], [200], 64), ([65, 1, 0, 20], [65, 90, 0, 333], 48)])
def test_attention_of_several_rows(n, ctx, page, Hq, Hkv, kind):
    attend(np.random.default_rng(Hq + sum(ctx)), n, ctx, page, kind, Hq, Hkv)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 20), (100, 0), (64, 64), (5000, 4), (50, 5000),
                                          (33, 16)])
@pytest.mark.parametrize("n,ctx,page", [([1], [300], 32), ([1, 1], [90, 513], 16), ([7, 2], [140, 260], 64),
                                        ([150], [280], 48)])
def test_window_and_sinks(n, ctx, page, window, sinks):
    attend(np.random.default_rng(window + sinks), n, ctx, page, INT8, 10, 2, window, sinks)


@pytest.mark.parametrize("n", [1, 9, 100])
def test_pages_that_the_window_has_left(n):
    """Their entries may be -1: the result is that of a cache that still holds them."""
    def drop(pages):
        first = (400 - n - 40 + 1) // 32
        pages[0, 1:first] = -1
    attend(np.random.default_rng(5), [n], [400], 32, E4M3, 10, 2, 40, 20, drop=drop)


@pytest.mark.parametrize("n", [1, 30])
def test_rows_that_see_nothing_give_zero(n):
    def drop(pages):
        pages[0] = [-1, 99, -5, 1 << 30] + [-1] * (pages.shape[1] - 4)
    got = attend(np.random.default_rng(6), [n, n], [100, 90], 32, INT8, 4, 2, drop=drop)
    assert np.all(got[:n] == 0) and np.any(got[n:] != 0)
    # a context shorter than its rows: the first rows have no token
    got = attend(np.random.default_rng(7), [n + 4, 2], [n, 33], 32, INT8, 4, 2)
    assert np.all(got[:4] == 0)


def test_missing_pages_in_between():
    def drop(pages):
        pages[0, 2], pages[1, 0], pages[0, 5] = -1, 1 << 20, -1
    attend(np.random.default_rng(8), [1, 1], [260, 150], 32, INT8, 16, 2, drop=drop)
    attend(np.random.default_rng(8), [33, 50], [260, 150], 32, INT8, 16, 2, drop=drop)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0, 1e-20])
def test_scales(scale):
    attend(np.random.default_rng(9), [1, 6], [70, 150], 16, INT8, 10, 2, scale=scale)
    attend(np.random.default_rng(9), [80], [150], 16, INT8, 10, 2, scale=scale)


@pytest.mark.parametrize("max_rows,max_ctx", [(1, 1), (5000, 1 << 20), (1, 1 << 20), (64, 10)])
def test_bounds_only_steer(max_rows, max_ctx):
    """max_rows and max_ctx choose a kernel and its split, not the result."""
    attend(np.random.default_rng(10), [40, 1, 3], [333, 1, 90], 32, INT8, 10, 2, max_rows=max_rows, max_ctx=max_ctx)


@pytest.mark.parametrize("n,ctx,Hq,Hkv,page", [([1], [20011], 40, 8, 64), ([1] * 9, [3000 + 501 * i for i in range(9)],
                                               16, 2, 16), ([5, 16], [9001, 4100], 10, 2, 32),
                                               ([300], [5000], 4, 1, 128)])
def test_long_contexts(n, ctx, Hq, Hkv, page):
    attend(np.random.default_rng(12), n, ctx, page, INT8, Hq, Hkv)


def test_huge_and_tiny_values():
    """Queries and values far from 1: the result is that of the scaled inputs,
    and a key that outweighs all others by far gives its value."""
    rng = np.random.default_rng(13)
    Hq, Hkv, page, L = 10, 2, 32, 100
    c = random_cache(rng, INT8, Hkv, page, 5)
    pages = np.array([[3, 1, 0, 4]], np.int32)
    q = rng.standard_normal((1, Hq, D)).astype(np.float32)
    for qs, ks, vs in ((2.0 ** 60, 2.0 ** -60, 2.0 ** 90), (2.0 ** -80, 2.0 ** 80, 2.0 ** -100), (1e4, 1.0, 1.0)):
        cc = dict(c, k_scales=(c["k_scales"] * ks).astype(np.float32), v_scales=(c["v_scales"] * vs).astype(np.float32))
        dev = device_cache(cc, INT8)
        ref = paged.attention(q * np.float32(qs), [0, 1], [L], pages, cc, INT8)
        out = torch.empty(1, Hq, D, device="cuda")
        tern.tern_attention_paged(to_dev(q * np.float32(qs)), tern.PagedBatch(i32([0, 1]), i32([L]), i32(pages), 1, 1, L),
                                  dev, out, tern.attention_paged_workspace(Hq, dev))
        k_ref, v_ref, _ = paged.values([0, L], [L], pages, cc, INT8)
        tol = bound((q * np.float32(qs)).astype(np.float64), k_ref.astype(np.float64), v_ref, D ** -0.5, L)
        assert np.all(np.abs(out.cpu().numpy() - ref) <= tol)


# ---------------------------------------------------------------- as they are used
@pytest.mark.parametrize("kind", [INT8, E4M3])
def test_prefill_verify_and_decode_in_one_graph_each(kind):
    """Prompts appended and attended, then tokens one by one through one
    captured graph whose lengths live on the device, against the oracle's cache
    and attention; the last steps of a sequence cross a page."""
    rng = np.random.default_rng(20)
    Hq, Hkv, page, window, sinks = 10, 2, 32, 50, 3
    prompts = [61, 5, 90]
    steps = 5
    total = [p + steps for p in prompts]
    pages, n_pages = page_table(rng, total, page)
    ref = random_cache(rng, kind, Hkv, page, n_pages)
    dev = device_cache(ref, kind)
    table = paged.rope_table(10000.0, D, 200)
    plan = tern.RopePlan(to_dev(table))
    ws = tern.attention_paged_workspace(Hq, dev)
    dpages = i32(pages)

    def check(out, q_ref, start, ctx):
        want = paged.attention(q_ref, start, ctx, pages, ref, kind, window, sinks)
        k_ref, v_ref, _ = paged.values(np.concatenate([[0], np.cumsum(ctx)]), ctx, pages, ref, kind)
        same_cache(dev, ref)
        err = np.abs(out.cpu().numpy() - want)
        assert np.all(err <= bound(q_ref, k_ref, v_ref, D ** -0.5, max(ctx))), float(err.max())

    def rows(n):
        qkv = rng.standard_normal((sum(n), (Hq + 2 * Hkv) * D)).astype(np.float32)
        return qkv, [qkv[:, a * D:b * D].reshape(-1, b - a, D) for a, b in
                     ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]

    def views(t):
        return [t[:, a * D:b * D].view(t.shape[0], b - a, D) for a, b in
                ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]

    start = np.concatenate([[0], np.cumsum(prompts)])
    qkv, host = rows(prompts)
    pos = np.concatenate([np.arange(p) for p in prompts])[None].astype(np.int32)
    batch = tern.PagedBatch(i32(start), i32(prompts), dpages, sum(prompts), max(prompts), max(prompts))
    q, k, v = views(to_dev(qkv))
    out = torch.empty(sum(prompts), Hq, D, device="cuda")
    tern.tern_kv_append_paged(q, k, v, to_dev(pos), plan, batch, dev, q)
    tern.tern_attention_paged(q, batch, dev, out, ws, window=window, sinks=sinks)
    q_ref, _ = paged.append(*host, pos, table, start, prompts, pages, ref, kind)
    check(out, q_ref, start, prompts)

    B = len(prompts)
    one = np.arange(B + 1)
    buf = torch.zeros(B, (Hq + 2 * Hkv) * D, device="cuda")
    dpos, dctx, out = i32(np.zeros((1, B))), i32(np.ones(B)), torch.empty(B, Hq, D, device="cuda")
    batch = tern.PagedBatch(i32(one), dctx, dpages, B, 1, max(total))
    q, k, v = views(buf)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    scratch = device_cache(ref, kind)
    with torch.cuda.stream(side):  # first calls outside the capture, on a cache of their own
        tern.tern_kv_append_paged(q, k, v, dpos, plan, batch, scratch, q)
        tern.tern_attention_paged(q, batch, scratch, out, ws, window=window, sinks=sinks)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tern.tern_kv_append_paged(q, k, v, dpos, plan, batch, dev, q)
        tern.tern_attention_paged(q, batch, dev, out, ws, window=window, sinks=sinks)
    for step in range(steps):
        ctx = [p + step + 1 for p in prompts]
        qkv, host = rows([1] * B)
        qkv *= np.float32(1.0 + step)
        pos = np.array([[c - 1 for c in ctx]], np.int32)
        buf.copy_(to_dev(qkv))
        dpos.copy_(to_dev(pos))
        dctx.copy_(i32(ctx))
        graph.replay()
        q_ref, _ = paged.append(*host, pos, table, one, ctx, pages, ref, kind)
        check(out, q_ref, one, ctx)


def test_buffers_of_another_kind_are_refused():
    cache = tern.PagedCache.empty(INT8, 1, D, 16, 2)
    batch = tern.PagedBatch(i32([0, 1]), i32([1]), i32([[0]]), 1, 1, 1)
    q = torch.zeros(1, 1, D, device="cuda")
    ws = tern.attention_paged_workspace(1, cache)
    with pytest.raises(ValueError):
        tern.tern_attention_paged(q.cpu(), batch, cache, torch.empty_like(q), ws)
    with pytest.raises(AssertionError):
        tern.tern_attention_paged(q.half(), batch, cache, torch.empty_like(q), ws)
    with pytest.raises(AssertionError):
        tern.tern_attention_paged(q, tern.PagedBatch(i32([0, 1]).long(), i32([1]), i32([[0]]), 1, 1, 1), cache,
                                  torch.empty_like(q), ws)
    with pytest.raises(tern.TernError):
        tern.tern_attention_paged(q, batch, cache, torch.empty_like(q), ws, window=-1)
    with pytest.raises(tern.TernError):
        tern.tern_attention_paged(q, batch, cache, q, ws)
