"""Plain numpy forms of the rotary embedding and the paged 8-bit KV cache.

TEST INFRASTRUCTURE, like the rest of this folder: nothing is shared with the
CUDA library.  The rotation and the quantisation are fp32 steps rounded one by
one (their results are unique); the attention is in 64 bits.

The cache is a dict of arrays: k_codes, v_codes uint8 [pages, Hkv, page, D] and
k_scales, v_scales fp32 [pages, Hkv, page / 16].
"""
from __future__ import annotations

import numpy as np

INT8, E4M3 = 0, 1
BLOCK = 16


def rope_table(theta: float, rot: int, n_pos: int, scale: float = 1.0) -> np.ndarray:
    f = theta ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    a = np.arange(n_pos, dtype=np.float64)[:, None] * scale * f
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def rope(x, pos, table, sections=None, interleaved=False, inverse=False):
    """x fp32 [T, H, D], pos [axes, T]; rows with a position outside the table give 0."""
    x = np.asarray(x, np.float32)
    T, H, D = x.shape
    n_pos, half = table.shape[:2]
    sections = [half] if sections is None else sections
    y = np.zeros_like(x)
    bad = 0
    for t in range(T):
        p = [int(pos[a, t]) for a in range(len(sections))]
        if any(v < 0 or v >= n_pos for v in p):
            bad += 1
            continue
        c, s = np.empty(half, np.float32), np.empty(half, np.float32)
        at = 0
        for a, k in enumerate(sections):
            c[at:at + k], s[at:at + k] = table[p[a], at:at + k, 0], table[p[a], at:at + k, 1]
            at += k
        if inverse:
            s = -s
        y[t] = x[t]
        i = np.arange(half)
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[t][:, lo] = x[t][:, lo] * c - x[t][:, hi] * s
        y[t][:, hi] = x[t][:, hi] * c + x[t][:, lo] * s
    return y, bad


_E4M3 = np.array([(-1.0 if b & 128 else 1.0) * ((b & 7) * 2.0 ** -9 if not (b >> 3) & 15 else
                                               (8 + (b & 7)) * 2.0 ** (((b >> 3) & 15) - 10)) for b in range(256)])
_E4M3[[127, 255]] = np.nan


def to_codes(y, kind):
    """fp32 -> codes: int8 half to even, or e4m3 to nearest even, saturating."""
    y = np.asarray(y, np.float32)
    if kind == INT8:
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(y.astype(np.float64)), 448.0)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6) - 3)  # spacing of the codes at a
    a = np.rint(a / step) * step
    code = np.searchsorted(_E4M3[:127], a).astype(np.uint8)
    return code | np.where(np.signbit(y), 128, 0).astype(np.uint8)


def from_codes(c, kind):
    c = np.asarray(c, np.uint8)
    return c.view(np.int8).astype(np.float32) if kind == INT8 else _E4M3[c].astype(np.float32)


def pow2_scale(amax: float, kind) -> np.float32:
    top = 127.0 if kind == INT8 else 448.0
    for e in range(-100, 121):
        if amax <= top * 2.0 ** e:
            return np.float32(2.0 ** e)
    return np.float32(2.0 ** 120)


def _page(pages, n_pages, b, tok, page):
    e = tok // page
    if tok < 0 or e >= pages.shape[1] or not 0 <= pages[b, e] < n_pages:
        return -1
    return int(pages[b, e])


def append(q, k, v, pos, table, row_start, ctx, pages, cache, kind, sections=None, interleaved=False, inverse=False):
    """q rotated, and the cache (in place) with the rotated k and v; the count of refused rows."""
    kr, _ = rope(k, pos, table, sections, interleaved, inverse)
    q_out, _ = rope(q, pos, table, sections, interleaved, inverse)
    n_pos = table.shape[0]
    axes = 1 if sections is None else len(sections)
    n_pages, Hkv, page, D = cache["k_codes"].shape
    bad = 0
    for b in range(len(ctx)):
        first = int(ctx[b]) - int(row_start[b + 1] - row_start[b])
        tok = np.arange(first, int(ctx[b]))
        for blk in np.unique(tok // BLOCK):
            mine = tok[tok // BLOCK == blk]
            rows = mine - first + int(row_start[b])
            pg = _page(pages, n_pages, b, int(mine[0]), page)
            ok = np.all([(pos[a, rows] >= 0) & (pos[a, rows] < n_pos) for a in range(axes)], 0)
            bad += len(rows) if pg < 0 else int((~ok).sum())
            if pg < 0:
                continue
            slot = mine % page
            base = int(blk) * BLOCK % page
            for x, name in ((kr, "k"), (v, "v")):
                for g in range(Hkv):
                    new = np.where(ok[:, None], x[rows, g], np.float32(0))
                    s = pow2_scale(float(np.abs(new).max()), kind)
                    at = cache[name + "_scales"][pg, g]
                    codes = cache[name + "_codes"][pg, g]
                    if slot[0] > base:
                        old = at[base // BLOCK]
                        s = max(old, s)
                        kept = from_codes(codes[base:slot[0]], kind) * np.float32(old / s)
                        codes[base:slot[0]] = to_codes(kept, kind)
                    codes[slot] = to_codes(new * np.float32(1.0 / s), kind)
                    at[base // BLOCK] = s
    return q_out, bad


def values(row_start, ctx, pages, cache, kind):
    """K and V values [T, Hkv, D] of the rows' tokens, and the rows without a page."""
    n_pages, Hkv, page, D = cache["k_codes"].shape
    T = int(row_start[-1])
    out = [np.zeros((T, Hkv, D), np.float32) for _ in range(2)]
    bad = 0
    for b in range(len(ctx)):
        for t in range(int(row_start[b]), int(row_start[b + 1])):
            tok = int(ctx[b]) - int(row_start[b + 1]) + t
            pg = _page(pages, n_pages, b, tok, page)
            if pg < 0:
                bad += 1
                continue
            for o, name in zip(out, "kv"):
                o[t] = (from_codes(cache[name + "_codes"][pg, :, tok % page], kind)
                        * cache[name + "_scales"][pg, :, tok % page // BLOCK, None])
    return out[0], out[1], bad


def attention(q, row_start, ctx, pages, cache, kind, window=0, sinks=0, scale=None):
    """64-bit attention [T, Hq, D]; a row that sees nothing gives 0."""
    T, Hq, D = q.shape
    n_pages, Hkv, page, _ = cache["k_codes"].shape
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros((T, Hq, D))
    for b in range(len(ctx)):
        L, n = int(ctx[b]), int(row_start[b + 1] - row_start[b])
        if n == 0 or L <= 0:
            continue
        toks = np.array([j for j in range(L) if _page(pages, n_pages, b, j, page) >= 0], np.int64)
        if not len(toks):
            continue
        pg = np.array([_page(pages, n_pages, b, int(j), page) for j in toks])
        kk, vv = (from_codes(cache[x + "_codes"][pg, :, toks % page], kind).astype(np.float64)
                  * cache[x + "_scales"][pg, :, toks % page // BLOCK][..., None] for x in "kv")
        for r in range(n):
            i = L - n + r
            see = toks <= i
            if window:
                see &= (toks > i - window) | (toks < sinks)
            if i < 0 or not see.any():
                continue
            t = int(row_start[b]) + r
            for h in range(Hq):
                g = h * Hkv // Hq
                x = kk[see, g] @ q[t, h].astype(np.float64) * scale
                w = np.exp(x - x.max())
                out[t, h] = (w / w.sum()) @ vv[see, g]
    return out
