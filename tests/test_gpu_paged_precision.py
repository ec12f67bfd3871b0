"""The paged attention's error, row by row against the 64-bit oracle: within
the bound counted from its arithmetic, and in the mean no more than a few times
that of the plain fp32 form on the same inputs (paged_bounds; on the host,
test_paged_bounds shows that both see a lost digit).  Also heads that rest on
their first token, by scores far above the rest and values far below it."""
import numpy as np
import pytest
import torch

from gpu_util import to_dev
from oracle import paged
from paged_bounds import RMS_FACTOR, border_query, bound_row, exponent, fp32_row, rms, softmax_row
from test_gpu_paged import D, E4M3, INT8, device_cache, i32, page_table
from ternary_weight_decode_b200 import tern

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def appended(rng, kind, Hkv, page, n_pages):
    """A cache of normal values, some channels of the keys stronger, as the append would hold them."""
    out = []
    for part in range(2):
        x = rng.standard_normal((n_pages, Hkv, page // 16, 16, D))
        if part == 0:
            x[..., ::37] *= 4.0
        x *= rng.random((n_pages, Hkv, page // 16, 1, 1)) + 0.25
        top = np.abs(x).max((-1, -2))
        s = np.exp2(np.ceil(np.log2(top / (127.0 if kind == INT8 else 448.0))))
        out += [paged.to_codes((x / s[..., None, None]).astype(np.float32), kind).reshape(n_pages, Hkv, page, D),
                s.astype(np.float32)]
    return dict(zip(("k_codes", "k_scales", "v_codes", "v_scales"), out))


def sequence(ref, pages, b, ctx, page, kind):
    """(K, V [Hkv, ctx, D], value scales [Hkv, ctx]) of a sequence, in 64 bits."""
    toks = np.arange(ctx)
    pg, slot = pages[b, toks // page], toks % page
    out = [paged.from_codes(ref[x + "_codes"][pg, :, slot], kind).astype(np.float64)
           * ref[x + "_scales"][pg, :, slot // 16][..., None] for x in "kv"]
    return out[0].swapaxes(0, 1), out[1].swapaxes(0, 1), ref["v_scales"][pg, :, slot // 16].T.astype(np.float64)


def run(q, start, ctx, pages, dev, kind, window=0, sinks=0):
    out = torch.full(q.shape, -2.0, device="cuda")
    n = int(np.diff(start).max())
    tern.tern_attention_paged(to_dev(q), tern.PagedBatch(i32(start), i32(ctx), i32(pages), len(q), n, int(max(ctx))), dev,
                              out, tern.attention_paged_workspace(q.shape[1], dev), window=window, sinks=sinks)
    assert tern.tern_device_error() == 0
    return out.cpu().numpy().astype(np.float64)


def most(plain, outs):
    """The root mean square that the errors are held to.  The second part: where one token has nearly all the weight, the
    plain form's weight is 1, its sum 1 and its output the token's value, without a rounding; the kernel rounds the sum of
    the digits, 1 / z (twice: the reciprocal and its factor) and their product: four roundings of up to 2^-24 of the
    output, each uniform, so 2^-24 * sqrt(4 / 3) and below 2^-23 in the mean."""
    return RMS_FACTOR * rms(plain) + 2.0 ** -23 * rms(outs)


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("n,ctx,Hq,Hkv,page,window,sinks,spread", [
    ([1, 1], [333, 1], 10, 2, 32, 0, 0, 1.5), ([1] * 5, [4096, 700, 129, 17, 2000], 5, 1, 16, 0, 0, 1.5),
    ([1] * 3, [900, 300, 70], 20, 2, 64, 0, 0, 5.0), ([7, 3], [260, 1100], 6, 2, 16, 100, 20, 1.5),
    ([40], [300], 8, 2, 32, 0, 0, 1.5), ([70], [2000], 2, 1, 64, 600, 4, 4.0), ([1], [20011], 8, 1, 64, 0, 0, 1.5)])
def test_every_row_is_within_its_bound(n, ctx, Hq, Hkv, page, window, sinks, spread, kind):
    rng = np.random.default_rng(sum(ctx) + Hq)
    pages, n_pages = page_table(rng, ctx, page)
    ref = appended(rng, kind, Hkv, page, n_pages)
    start = np.concatenate([[0], np.cumsum(n)])
    q = (rng.standard_normal((sum(n), Hq, D)) * spread).astype(np.float32)
    got = run(q, start, ctx, pages, device_cache(ref, kind), kind, window, sinks)
    plain, mine, outs = [], [], []
    for b, L in enumerate(ctx):
        K, V, s = sequence(ref, pages, b, L, page, kind)
        for r in range(n[b]):
            i = L - n[b] + r
            j = np.arange(i + 1)
            see = j if not window else j[(j > i - window) | (j < sinks)]
            for h in range(Hq):
                g, row = h * Hkv // Hq, q[start[b] + r, h]
                out = softmax_row(row, K[g, see], V[g, see], SCALE)[2]
                err = got[start[b] + r, h] - out
                tol = bound_row(row, K[g, see], V[g, see], s[g, see], SCALE, kind)
                assert np.all(np.abs(err) <= tol), (b, r, h, np.abs(err).max(), tol.min())
                mine.append(err)
                outs.append(out)
                plain.append(fp32_row(row, K[g, see], V[g, see], SCALE) - out)
    assert rms(mine) <= most(plain, outs), (rms(mine), rms(plain))


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("ratio", [1.0, 1 / 16, 1 / 64])
@pytest.mark.parametrize("above", [24.0, 27.5, 28.5])
@pytest.mark.parametrize("B,ctx,window", [(148, 4096, 0), (3, 4096, 0), (148, 65536, 0), (20, 9000, 4096)])
def test_heads_that_rest_on_their_first_token(B, ctx, window, above, ratio, kind):
    """The first token's score lies 2^above over the others', its block's value scale is `ratio` of theirs.  B sequences
    share the pages, so that a CTA has whole items (148) or pieces of one."""
    rng = np.random.default_rng(int(above * 2) + ctx)
    Hq, page, sinks = 4, 64, 4 if window else 0
    n_pages = -(-ctx // page)
    ref = appended(rng, kind, 1, page, n_pages)
    pages = np.tile(rng.permutation(n_pages).astype(np.int32), (B, 1))
    first = int(pages[0, 0])
    ref["v_scales"][first, 0, 0] = np.float32(ratio) * ref["v_scales"].max()
    # a first key that no other resembles
    ref["k_codes"][first, 0, 0] = paged.to_codes((rng.choice([-1.0, 1.0], D) * 100).astype(np.float32), kind)
    ref["k_scales"][first, 0, 0] = np.float32(2.0 ** -4)
    dev = device_cache(ref, kind)
    K, V, s = (x[0] for x in sequence(ref, pages, 0, ctx, page, kind))
    # queries of small scores, and what brings the first token's to `above` (log2) over the largest of the others
    q = rng.standard_normal((Hq, D)) * 0.5
    along = K[0] / (K[0] @ K[0])
    for h in range(Hq):
        for _ in range(60):
            x = K @ q[h] * (SCALE * np.log2(np.e))
            q[h] += along * (above - (x[0] - x[1:].max())) / (SCALE * np.log2(np.e))
        assert abs(x[0] - x[1:].max() - above) < 0.01
    q = q.astype(np.float32)
    got = run(np.tile(q, (B, 1, 1)), np.arange(B + 1), [ctx] * B, pages, dev, kind, window, sinks)
    see = np.arange(ctx)
    if window:
        see = see[(see > ctx - 1 - window) | (see < sinks)]
    K, V, s = K[see], V[see], s[see]
    plain, mine, outs = [], [], []
    for h in range(Hq):
        x, p, out = softmax_row(q[h], K, V, SCALE)
        T = p * np.exp2(exponent(s))
        # the first tile's reference is the first token's; behind it references fall to the others'
        place = np.arange(len(see)) if not window else np.where(see < 16, see, see - see[see >= 16].min() // 16 * 16 + 16)
        tiles = np.where(place < 128, T.max(), T[place >= 128].max())
        tol = bound_row(q[h], K, V, s, SCALE, kind, tiles)
        err = got[:, h] - out
        assert np.all(np.abs(err) <= tol), (h, np.abs(err).max(), tol.min(), np.abs(out).max())
        outs.append(out / np.abs(out).max())
        mine.append(err / np.abs(out).max())
        plain.append((fp32_row(q[h], K, V, SCALE) - out) / np.abs(out).max())
    print("relative to the largest output: mine %.2e (rms %.2e), plain %.2e (rms %.2e)" % (
        np.abs(mine).max(), rms(mine), np.abs(plain).max(), rms(plain)))
    assert rms(mine) <= most(plain, outs), (rms(mine), rms(plain))


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("n,ctx", [(1, 100), (3, 2000), (30, 700)])
def test_a_key_that_outweighs_all_others_gives_its_value(n, ctx, kind):
    rng = np.random.default_rng(ctx)
    Hq, Hkv, page = 6, 2, 32
    pages, n_pages = page_table(rng, [ctx], page)
    ref = appended(rng, kind, Hkv, page, n_pages)
    q = (rng.standard_normal((n, Hq, D)) * 1e4).astype(np.float32)
    got = run(q, np.array([0, n]), [ctx], pages, device_cache(ref, kind), kind)
    K, V, s = sequence(ref, pages, 0, ctx, page, kind)
    alone = 0
    for r in range(n):
        for h in range(Hq):
            g, see = h * Hkv // Hq, ctx - n + r + 1
            x = np.sort(K[g, :see] @ q[r, h].astype(np.float64) * SCALE)
            if x[-1] - x[-2] < 40.0:   # e^-40 of the next key's value is below an fp32 step
                continue
            alone += 1
            v = V[g, int(np.argmax(K[g, :see] @ q[r, h].astype(np.float64)))]
            # one weight: its exponential divides out, its digits are off by 2^-20 at most; and the other tokens' weights,
            # below e^-40 of it each
            assert np.all(np.abs(got[r, h] - v) <= 2.0 ** -20 * np.abs(v) + see * np.exp(-40.0) * np.abs(V[g, :see]).max())
    assert alone >= n * Hq / 2


@pytest.mark.parametrize("rows", [1, 9, 40])
def test_queries_between_the_digits_steps(rows):
    """int8: a row whose largest element is just a power of two, the others half-way between the steps of 22 bits."""
    rng = np.random.default_rng(rows)
    q, signs = zip(*(border_query(rng) for _ in range(rows)))
    q = np.stack(q)[:, None]
    code = (100 * signs[0]).astype(np.int8)
    codes = np.zeros((1, 1, 48, D), np.int8)
    codes[0, 0, 0], codes[0, 0, 1:16] = code, -code
    ref = dict(k_codes=codes.view(np.uint8).copy(), k_scales=np.ones((1, 1, 3), np.float32), v_scales=np.ones((1, 1, 3), np.float32))
    codes[0, 0, 0], codes[0, 0, 1:16] = 100, -100
    ref["v_codes"] = codes.view(np.uint8)
    ctx = 2 + rows - 1   # row 0 sees two tokens, the others more of the second kind
    if rows > 1:
        ref["k_codes"][0, 0, 2:], ref["v_codes"][0, 0, 2:] = ref["k_codes"][0, 0, 1], ref["v_codes"][0, 0, 1]
    pages = np.array([[0]], np.int32)
    got = run(q, np.array([0, rows]), [ctx], pages, device_cache(ref, INT8), INT8)
    K, V, s = (x[0] for x in sequence(ref, pages, 0, ctx, 48, INT8))
    for r in range(rows):
        see = 2 + r
        tol = bound_row(q[r, 0], K[:see], V[:see], s[:see], SCALE, INT8)
        assert np.all(np.abs(got[r, 0] - softmax_row(q[r, 0], K[:see], V[:see], SCALE)[2]) <= tol)


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("B,rows,Hq,ctx", [(148, 1, 4, 1500), (2, 1, 12, 700), (40, 5, 3, 1300), (1, 60, 2, 900), (148, 30, 1, 600)])
@pytest.mark.parametrize("order", ["zeros first", "zeros between", "rising", "falling", "mixed"])
def test_value_scales_far_apart(order, B, rows, Hq, ctx, kind):
    """Values of tiles (or blocks) that differ by up to 2^26, and blocks of zeros, whose scale is the append's least."""
    rng = np.random.default_rng(ctx + rows)
    page = 128
    n_pages = -(-ctx // page)
    ref = appended(rng, kind, 1, page, n_pages)
    pages = np.tile(np.arange(n_pages, dtype=np.int32), (B, 1))
    t = np.arange(n_pages)[:, None] + np.zeros(8, int)
    shift = {"zeros first": np.zeros_like(t), "zeros between": np.zeros_like(t), "rising": np.minimum(26, 5 * t),
             "falling": -np.minimum(26, 5 * t), "mixed": rng.integers(-13, 14, t.shape)}[order]
    ref["v_scales"][:, 0] *= np.exp2(shift).astype(np.float32)
    zero = {"zeros first": t < 2, "zeros between": t % 3 == 1, "mixed": rng.random(t.shape) < 0.2}.get(order, t < 0)
    ref["v_scales"][:, 0][zero] = 2.0 ** -100
    ref["v_codes"].reshape(n_pages, 8, 16, D)[zero] = 0
    dev = device_cache(ref, kind)
    one = (rng.standard_normal((rows, Hq, D)) * 1.5).astype(np.float32)
    start = np.arange(B + 1) * rows
    got = run(np.tile(one, (B, 1, 1)), start, [ctx] * B, pages, dev, kind).reshape(B, rows, Hq, D)
    K, V, s = (x[0] for x in sequence(ref, pages, 0, ctx, page, kind))
    for r in range(0, rows, max(1, rows // 8)):
        see = ctx - rows + r + 1
        for h in range(Hq):
            out = softmax_row(one[r, h], K[:see], V[:see], SCALE)[2]
            tol = bound_row(one[r, h], K[:see], V[:see], s[:see], SCALE, kind)
            err = np.abs(got[:, r, h] - out)
            assert np.all(err <= tol), (r, h, err.max(), tol.min(), np.abs(out).max())


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("above", [60.0, 130.0, 300.0])
@pytest.mark.parametrize("zeros", [16, 128, 256])
@pytest.mark.parametrize("B", [1, 148])
def test_zeros_far_above_the_rest(B, zeros, above, kind):
    """A first token 2^above over the others whose block, or whose first tiles, have values of 0: the output is finite, and
    nothing but what the others' weights leave of their values."""
    rng = np.random.default_rng(zeros)
    page, ctx, Hq = 128, 1000, 3
    n_pages = -(-ctx // page)
    ref = appended(rng, kind, 1, page, n_pages)
    flat = ref["v_codes"].reshape(n_pages * page, D)
    flat[:zeros] = 0
    ref["v_scales"].reshape(-1)[:zeros // 16] = 2.0 ** -100
    ref["k_codes"][0, 0, 0] = paged.to_codes((rng.choice([-1.0, 1.0], D) * 100).astype(np.float32), kind)
    ref["k_scales"][0, 0, 0] = np.float32(2.0 ** -4)
    pages = np.tile(np.arange(n_pages, dtype=np.int32), (B, 1))
    K, V, s = (x[0] for x in sequence(ref, pages, 0, ctx, page, kind))
    q = rng.standard_normal((Hq, D)) * 0.5
    for h in range(Hq):
        for _ in range(60):
            x = K @ q[h] * (SCALE * np.log2(np.e))
            q[h] += K[0] / (K[0] @ K[0]) * (above - (x[0] - x[1:].max())) / (SCALE * np.log2(np.e))
    q = q.astype(np.float32)
    got = run(np.tile(q, (B, 1, 1)), np.arange(B + 1), [ctx] * B, pages, device_cache(ref, kind), kind)
    assert np.all(np.isfinite(got))
    # a weight 2^-above of the first's, at most; it may be off by all of itself where it lies below what is kept
    most = min(1.0, ctx * 2.0 ** (1 - above)) * np.abs(V).max()
    assert np.all(np.abs(got) <= most)
