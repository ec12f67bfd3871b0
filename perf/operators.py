"""The paged 8-bit KV cache's operators and the sizes they are measured at.

``run`` makes one pass through one operator: the rotary embedding (``rope``),
the append to the paged cache (``append``) or the attention over it
(``attention``).  With ``own`` false it is the plain form, elementary torch
operations in fp32; with ``own`` true it is the call a user of the package
makes.  The 40 query / 8 KV heads of 128 are the attention of the 27B-shaped
decode step; the other head counts are generic.

A case's row counts and context lengths follow from its own numbers (``lens``
seeds them), its values from the seed given to ``prepare``.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16  # tokens that share a scale, per KV head
INT8, E4M3 = 0, 1
THETA = 1000000.0


def listed():
    rope = dict(op="rope", D=128, rot=128, interleaved=False, inverse=False, strided=True)
    app = dict(op="append", Hq=40, Hkv=8, kind=INT8, page=64, axes=1, ragged=False, lens=0)
    att = dict(op="attention", Hq=40, Hkv=8, kind=INT8, page=64, window=0, sinks=0, ragged=False, lens=0)
    return [
        # the smallest call: q and k heads of one decoded token
        dict(rope, name="rope_1_token", T=1, H=48, axes=1),
        # a prefill batch of text and image tokens (three position axes), in place in the QKV rows
        dict(rope, name="rope_2048_3axes", T=2048, H=48, axes=3),
        # partial rotation of interleaved pairs, an odd row count, contiguous rows
        dict(rope, name="rope_777_partial", T=777, H=32, rot=64, axes=1, interleaved=True, strided=False),
        # batch-1 decode: one token into a cache of 4096
        dict(app, name="append_decode_1", B=1, rows=1, ctx=4096),
        # a prompt of 4096 tokens, positions on three axes
        dict(app, name="append_prefill_4096", B=1, rows=4096, ctx=4096, axes=3),
        # a serving batch with drafted tokens: ragged rows, small pages, fp8 codes
        dict(app, name="append_ragged_e4m3", B=33, rows=16, ctx=2500, kind=E4M3, page=32, ragged=True, lens=5),
        # batch-1 decode at a middling context
        dict(att, name="decode_1_4096", B=1, rows=1, ctx=4096),
        # batch-1 decode at 64K tokens
        dict(att, name="decode_1_65536", B=1, rows=1, ctx=65536),
        # a serving batch of uneven contexts, fp8 codes
        dict(att, name="decode_24_ragged_e4m3", B=24, rows=1, ctx=20011, kind=E4M3, page=16, ragged=True, lens=7),
        # long contexts behind a sliding window with first tokens that stay visible
        dict(att, name="decode_16_window_sinks", B=16, rows=1, ctx=32768, window=4096, sinks=4),
        # 16 drafted tokens each for three sequences
        dict(att, name="verify_3x16", B=3, rows=16, ctx=8191),
        # the second half of a prompt, causal over what is cached
        dict(att, name="prefill_2048_of_4096", B=1, rows=2048, ctx=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "attention", "attention", "attention"])
    if op == "rope":
        D = rng.choice([64, 128, 128, 256])
        rot = rng.choice([D, D, D // 2])
        H = rng.choice([1, 7, 8, 16, 40, 48])
        T = min(_log(rng, 1, 4096), 12000000 // (H * D))
        return dict(op=op, T=T, H=H, D=D, rot=rot, axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.random() < 0.4, inverse=rng.random() < 0.3, strided=rng.random() < 0.5)
    Hq, Hkv = rng.choice([(40, 8), (40, 8), (32, 8), (8, 8), (16, 2), (7, 1), (24, 2)])
    base = dict(op=op, Hq=Hq, Hkv=Hkv, kind=rng.choice([INT8, INT8, E4M3]),
                page=rng.choice([16, 32, 48, 64, 128]), ragged=rng.random() < 0.6, lens=rng.randrange(1 << 20))
    if op == "append":
        B = _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, 4096 // B))
        return dict(base, B=B, rows=rows, ctx=rows + _log(rng, 1, 4096) - 1, axes=rng.choice([1, 1, 3]))
    form = rng.choice(["decode", "decode", "verify", "prefill"])
    if form == "decode":
        B, rows = _log(rng, 1, 64), 1
    elif form == "verify":
        B, rows = _log(rng, 1, 16), rng.randint(2, 16)
    else:
        B, rows = _log(rng, 1, 4), _log(rng, 17, 1024)
    most = min(65536, 262144 // B) if rows == 1 else 16384 // B if rows <= 16 else 8192 // B
    ctx = max(rows, _log(rng, 40, most))
    window = 0 if rng.random() < 0.5 else _log(rng, 16, 4096)
    sinks = rng.choice([0, 1, 4, 4, 20, 64]) if window else 0
    return dict(base, B=B, rows=rows, ctx=ctx, window=window, sinks=sinks)


# ------------------------------------------------------------- sizes of a case
def _lens(case):
    """Rows and context (those rows included) of each sequence."""
    B, rows, ctx = case["B"], case["rows"], case["ctx"]
    if not case["ragged"]:
        return [rows] * B, [ctx] * B
    r = random.Random(case["lens"])
    n = [rows] + [r.randint(1, rows) for _ in range(B - 1)]
    c = [ctx] + [r.randint(max(n[b], ctx // 8), max(n[b], ctx)) for b in range(1, B)]
    return n, c


def _visible(case, n, ctx):
    """(tokens that any row of the sequence sees, pairs of a row and a token it sees)."""
    W, S = case["window"], case["sinks"]
    p = np.arange(ctx - n, ctx, dtype=np.int64)
    if not W:
        return ctx, int((p + 1).sum())
    low = np.maximum(p - W + 1, 0)
    return ctx - int(low[0]) + min(S, int(low[0])), int((p + 1 - low + np.minimum(S, low)).sum())


def work(case):
    if case["op"] == "rope":
        x = 4 * case["T"] * case["H"] * case["D"]
        return {"bytes": 2 * x + case["T"] * (4 * case["axes"] + 4 * case["rot"]),
                "flops": 3 * case["T"] * case["H"] * case["rot"]}
    n, c = _lens(case)
    Hq, Hkv, D, T = case["Hq"], case["Hkv"], 128, sum(n)
    if case["op"] == "append":
        blocks = sum((c[b] - 1) // BLOCK - (c[b] - n[b]) // BLOCK + 1 for b in range(len(n)))
        seen = sum(c[b] - (c[b] - n[b]) // BLOCK * BLOCK for b in range(len(n)))
        return {"bytes": T * (2 * Hq + 2 * Hkv) * D * 4 + T * 2 * Hkv * D + blocks * 2 * Hkv * 4
                + T * (4 * case["axes"] + 4 * D)
                # the touched blocks read back as values
                + seen * 2 * Hkv * D * (1 + 4) + blocks * 2 * Hkv * 4,
                "flops": 3 * T * (Hq + Hkv) * D + 4 * T * Hkv * D}
    seen = [_visible(case, n[b], c[b]) for b in range(len(n))]
    tokens, pairs = sum(s[0] for s in seen), sum(s[1] for s in seen)
    return {"bytes": 2 * T * Hq * D * 4 + tokens * Hkv * 2 * (D + 4 / BLOCK) + tokens // case["page"] * 4,
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------- inputs
def _pow2_scale(amax, kind):
    """The least power of two s (exponent -100..120) with amax <= s * the largest code."""
    m, e = torch.frexp(amax)
    top = 127 / 128 if kind == INT8 else 448 / 512
    e = e - (7 if kind == INT8 else 9) + (m > top).to(e.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(-100, 120)
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _codes(x, scale, kind):
    y = x / scale
    if kind == INT8:
        return y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, kind):
    return codes.view(torch.int8 if kind == INT8 else torch.float8_e4m3fn).float()


def _table(n_pos, rot):
    f = THETA ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _sections(pairs, axes):
    """Pairs of each axis: a quarter for the first of three, the rest halved."""
    if axes == 1:
        return [pairs]
    if axes == 2:
        return [pairs // 2, pairs - pairs // 2]
    h = (pairs - pairs // 4) // 2
    return [pairs - 2 * h, h, h]


def _cache(g, case, n_pages):
    """A cache whose pages hold quantised values: keys with a few strong channels, values without."""
    Hkv, page, D, kind = case["Hkv"], case["page"], 128, case["kind"]
    out = []
    for part in range(2):
        x = torch.randn(n_pages, Hkv, page // BLOCK, BLOCK, D, generator=g, device="cuda")
        if part == 0:
            x[..., ::37] *= 4.0
        x *= torch.rand(n_pages, Hkv, page // BLOCK, 1, 1, generator=g, device="cuda") + 0.25
        s = _pow2_scale(x.abs().amax((-1, -2)), kind)
        out += [_codes(x, s[..., None, None], kind).reshape(n_pages, Hkv, page, D), s]
    return out


def _pages(g, case, n, c):
    """Page table [B, ld], pages in random order, -1 where a sequence has none or every row's window has left it."""
    page = case["page"]
    per = [-(-x // page) for x in c]
    total = sum(per)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    idx = np.full((len(c), max(per)), -1, np.int64)
    at = 0
    for b, k in enumerate(per):
        idx[b, :k] = np.arange(at, at + k)
        if case.get("window"):
            first = max(0, c[b] - n[b] - case["window"] + 1) // page
            idx[b, min(-(-case["sinks"] // page), first):first] = -1
        at += k
    i = torch.from_numpy(idx).cuda()
    return torch.where(i >= 0, perm[i.clamp(min=0)], torch.full_like(i, -1).to(torch.int32)).contiguous(), total


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        wide = torch.randn(T, (H + 8) * D if case["strided"] else H * D, generator=g, device="cuda")
        s["x"] = wide[:, :H * D].view(T, H, D)
        s["y"] = torch.empty(T, H, D, device="cuda")
        s["n_pos"] = 8192
        s["table"] = _table(s["n_pos"], case["rot"])
        s["sections"] = _sections(case["rot"] // 2, case["axes"])
        s["pos"] = torch.randint(0, s["n_pos"], (case["axes"], T), generator=g, device="cuda", dtype=torch.int32)
        if own:
            from ternary_weight_decode_b200 import tern
            s["rope"] = tern.RopePlan(s["table"], s["sections"], interleaved=case["interleaved"],
                                      inverse=case["inverse"])
        return s
    n, c = _lens(case)
    T, Hq, Hkv, D = sum(n), case["Hq"], case["Hkv"], 128
    s["pages"], total = _pages(g, case, n, c)
    s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"] = _cache(g, case, total)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    s["row_start"] = torch.from_numpy(start).cuda()
    s["ctx"] = torch.tensor(c, dtype=torch.int32, device="cuda")
    s["T"], s["max_rows"], s["max_ctx"] = T, max(n), max(c)
    if own:
        from ternary_weight_decode_b200 import tern
        s["cache"] = tern.PagedCache(case["kind"], Hkv, D, case["page"], s["k_codes"], s["k_scales"],
                                     s["v_codes"], s["v_scales"])
        s["batch"] = tern.PagedBatch(s["row_start"], s["ctx"], s["pages"], T, s["max_rows"], s["max_ctx"])
    if case["op"] == "attention":
        s["q"] = 1.5 * torch.randn(T, Hq, D, generator=g, device="cuda")
        if own:
            s["out"] = torch.empty(T, Hq, D, device="cuda")
            s["ws"] = tern.attention_paged_workspace(Hq, s["cache"])
        return s
    # append: the rows as the QKV projection wrote them
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda")
    s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
    s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    s["k"][..., ::37] *= 4.0
    s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    s["n_pos"] = max(c) + 64
    s["table"] = _table(s["n_pos"], D)
    s["sections"] = _sections(D // 2, case["axes"])
    line = torch.cat([torch.arange(c[b] - n[b], c[b], device="cuda", dtype=torch.int32) for b in range(len(n))])
    s["pos"] = torch.stack([line] + [torch.randint(0, s["n_pos"], (T,), generator=g, device="cuda", dtype=torch.int32)
                                     for _ in range(case["axes"] - 1)]).contiguous()
    # the touched blocks of each sequence, to be read back as values
    seen = [c[b] - (c[b] - n[b]) // BLOCK * BLOCK for b in range(len(n))]
    s["T_read"] = sum(seen)
    s["read_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(seen)]).astype(np.int32)).cuda()
    if own:
        s["rope"] = tern.RopePlan(s["table"], s["sections"])
        s["read"] = tern.PagedBatch(s["read_start"], s["ctx"], s["pages"], s["T_read"], max(seen), s["max_ctx"])
        s["q_out"] = torch.empty(T, Hq, D, device="cuda")
        s["k_read"] = torch.empty(s["T_read"], Hkv, D, device="cuda")
        s["v_read"] = torch.empty(s["T_read"], Hkv, D, device="cuda")
    return s


# ------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "rope":
        return _plain_rope(s, s["x"], s["pos"], s["rot"], s["interleaved"], s["inverse"])
    return _plain_append(s) if s["op"] == "append" else _plain_attention(s)


def _run_own(s):
    from ternary_weight_decode_b200 import tern
    if s["op"] == "rope":
        tern.tern_rope(s["rope"], s["pos"], s["x"], s["y"])
        return s["y"]
    if s["op"] == "append":
        tern.tern_kv_append_paged(s["q"], s["k"], s["v"], s["pos"], s["rope"], s["batch"], s["cache"], s["q_out"])
        tern.tern_kv_read_paged(s["read"], s["cache"], s["k_read"], s["v_read"])
        return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"]}
    tern.tern_attention_paged(s["q"], s["batch"], s["cache"], s["out"], s["ws"], window=s["window"], sinks=s["sinks"])
    return s["out"]


def _plain_rope(s, x, pos, rot, interleaved, inverse):
    pairs = rot // 2
    i = torch.arange(pairs, device=x.device)
    bounds = torch.tensor(np.cumsum(s["sections"]), device=x.device)
    axis = torch.searchsorted(bounds, i, right=True)
    cs = s["table"][pos[axis].long().T, i]                    # [T, pairs, 2]
    c, sn = cs[..., 0][:, None], cs[..., 1][:, None]
    sn = -sn if inverse else sn
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :pairs], x[..., pairs:rot])
    u, w = a * c - b * sn, b * c + a * sn
    y = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s):
    Hkv, page, kind, D = s["Hkv"], s["page"], s["kind"], 128
    q = _plain_rope(s, s["q"], s["pos"], D, False, False)
    k = _plain_rope(s, s["k"], s["pos"], D, False, False)
    start, ctx, pages = s["row_start"].long(), s["ctx"].long(), s["pages"].long()
    first = ctx - (start[1:] - start[:-1])                    # position of the first new token
    j0, j1 = first // BLOCK, (ctx - 1) // BLOCK
    nb = (s["max_rows"] + BLOCK - 2) // BLOCK + 1
    blk = torch.minimum(j0[:, None] + torch.arange(nb, device=q.device), j1[:, None])   # [B, nb], the last one repeated
    tok = blk[..., None] * BLOCK + torch.arange(BLOCK, device=q.device)                 # [B, nb, 16]
    new = (tok >= first[:, None, None]) & (tok < ctx[:, None, None])
    old = (tok < first[:, None, None])
    row = (start[:-1, None, None] + tok - first[:, None, None]).clamp(0, s["T"] - 1)
    at = torch.gather(pages, 1, blk * BLOCK // page), blk * BLOCK % page // BLOCK       # page, block in it
    for x, codes, scales in ((k, s["k_codes"], s["k_scales"]), (s["v"], s["v_codes"], s["v_scales"])):
        x = torch.where(new[..., None, None], x[row], torch.zeros((), device=q.device)).transpose(2, 3)  # [B, nb, Hkv, 16, D]
        held = codes.view(-1, Hkv, page // BLOCK, BLOCK, D)
        c0, s0 = held[at[0], :, at[1]], scales[at[0], :, at[1]]                         # [B, nb, Hkv, 16, D], [B, nb, Hkv]
        need = _pow2_scale(x.abs().amax((-1, -2)), kind)
        s1 = torch.where(old.any(-1)[..., None], torch.maximum(need, s0), need)
        kept = _codes(_values(c0, kind) * s0[..., None, None], s1[..., None, None], kind)
        c1 = torch.where(new[:, :, None, :, None], _codes(x, s1[..., None, None], kind),
                         torch.where(old[:, :, None, :, None], kept, c0))
        held[at[0], :, at[1]] = c1
        scales[at[0], :, at[1]] = s1
    # the touched blocks as values
    r = torch.arange(s["T_read"], device=q.device)
    seq = torch.searchsorted(s["read_start"][1:].long(), r, right=True)
    t = ctx[seq] - s["read_start"][1:].long()[seq] + r
    p = pages[seq, t // page]
    kk = _values(s["k_codes"][p, :, t % page], kind) * s["k_scales"][p, :, t % page // BLOCK][..., None]
    vv = _values(s["v_codes"][p, :, t % page], kind) * s["v_scales"][p, :, t % page // BLOCK][..., None]
    return {"q": q, "k": kk, "v": vv}


def _plain_attention(s):
    Hq, Hkv, page, kind, D = s["Hq"], s["Hkv"], s["page"], s["kind"], 128
    G, n, L, T = Hq // Hkv, s["max_rows"], s["max_ctx"], s["T"]
    start, ctx = s["row_start"].long(), s["ctx"].long()
    B = ctx.numel()
    t = torch.arange(L, device="cuda")
    p = s["pages"].long()[:, t // page]                       # [B, L]
    held = (p >= 0) & (t < ctx[:, None])
    p = p.clamp(min=0)
    k = _values(s["k_codes"][p, :, t % page], kind) * s["k_scales"][p, :, t % page // BLOCK][..., None]  # [B, L, Hkv, D]
    v = _values(s["v_codes"][p, :, t % page], kind) * s["v_scales"][p, :, t % page // BLOCK][..., None]
    rows = start[:-1, None] + torch.arange(n, device="cuda")  # [B, n], past the sequence's own rows: padding
    i = rows + (ctx - start[1:])[:, None]                     # position of each row
    q = s["q"][rows.clamp(max=T - 1)].view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    see = held[:, None] & (t <= i[..., None])
    if s["window"]:
        see &= (t > i[..., None] - s["window"]) | (t < s["sinks"])
    x = (q @ k.permute(0, 2, 3, 1)).view(B, Hkv, n, G, L) * (1.0 / math.sqrt(D))
    x.masked_fill_(~see[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    z = x.sum(-1, keepdim=True)
    o = (x.view(B, Hkv, n * G, L) @ v.transpose(1, 2)).view(B, Hkv, n, G, D)
    o = torch.where(z > 0, o / z, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    seq = torch.searchsorted(start[1:], torch.arange(T, device="cuda"), right=True)
    return o[seq, torch.arange(T, device="cuda") - start[seq]]


# ------------------------------------------------------------- 64-bit values
def _exact_rotation(x, table, pos, rot, sections, interleaved, sign):
    """Each pair as a complex number times c + i s of its axis' position."""
    x = x.double()
    z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else torch.complex(x[..., :rot // 2], x[..., rot // 2:rot])
    table = table.double()
    turn = []
    at = 0
    for a, k in enumerate(sections):
        e = table[pos[a].long(), at:at + k]
        turn.append(torch.complex(e[..., 0], sign * e[..., 1]))
        at += k
    z = z * torch.cat(turn, -1)[:, None]
    y = x.clone()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotation(s["x"], s["table"], s["pos"], case["rot"], s["sections"], case["interleaved"],
                               -1.0 if case["inverse"] else 1.0)
    if case["op"] == "append":
        # what the cache holds is decided by roundings of the fp32 rotation: no 64-bit value
        return {"q": _exact_rotation(s["q"], s["table"], s["pos"], 128, s["sections"], False, 1.0), "k": None, "v": None}
    n, c = _lens(case)
    Hq, Hkv, page, D = case["Hq"], case["Hkv"], case["page"], 128
    out = torch.zeros(sum(n), Hq, D, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(len(n)):
        table = s["pages"][b, : -(-c[b] // page)].long()
        pair = []
        for part in ("k", "v"):
            code, scale = s[part + "_codes"][table.clamp(min=0)], s[part + "_scales"][table.clamp(min=0)]
            x = _values(code, case["kind"]).double() * scale.double().repeat_interleave(BLOCK, -1)[..., None]
            pair.append(x.transpose(0, 1).reshape(Hkv, -1, D)[:, :c[b]])
        j = torch.arange(c[b], device="cuda")
        for r0 in range(0, n[b], 256):
            r1 = min(n[b], r0 + 256)
            i = torch.arange(c[b] - n[b] + r0, c[b] - n[b] + r1, device="cuda")[:, None]
            see = (j <= i) & (table >= 0).repeat_interleave(page)[:c[b]]
            if case["window"]:
                see = see & ((i - j < case["window"]) | (j < case["sinks"]))
            for h in range(Hq):
                x = s["q"][at + r0:at + r1, h].double() @ pair[0][h * Hkv // Hq].T / math.sqrt(D)
                w = torch.softmax(x.masked_fill(~see, -math.inf), -1)
                out[at + r0:at + r1, h] = torch.nan_to_num(w, nan=0.0) @ pair[1][h * Hkv // Hq]
        at += n[b]
    return out
