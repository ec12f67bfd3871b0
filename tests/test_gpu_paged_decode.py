"""The decode step with its attention over the paged 8-bit KV cache.

Eager steps record each layer's QKV output and attention; the oracle appends
the recorded rows to its own cache (equal bit for bit) and attends over it.  A
captured graph, whose lengths advance on the device, repeats the eager steps."""
import numpy as np
import pytest
import torch

from oracle import paged
from ternary_weight_decode_b200 import decode, synth, tern
from test_gpu_paged import bound

pytestmark = pytest.mark.gpu
H, QKV, F, LAYERS = 512, 1024, 768, 2   # 4 query heads, 2 KV heads of 128


def model(M, mode, **att):
    m = decode.DecodeModel(tern.TERN_FMT_BASE3, LAYERS, M=M, hidden=H, qkv=QKV, ffn=F, mode=mode,
                           attention=decode.PagedAttention(**att)).build()
    assert (m.attention.Hq, m.attention.Hkv) == (4, 2)
    return m


def start(m, rng, ctx):
    """The same random cache contents and input on every call with the same rng state."""
    x = rng.standard_normal((m.M, H)).astype(np.float32)
    m.x.copy_(torch.from_numpy(x))
    for c in m.attention.caches:
        for t in (c.k_codes, c.v_codes):
            codes = rng.integers(0, 120, tuple(t.shape), dtype=np.uint8)
            t.copy_(torch.from_numpy(codes))
        for t in (c.k_scales, c.v_scales):
            t.copy_(torch.from_numpy(np.exp2(rng.integers(-9, -5, tuple(t.shape))).astype(np.float32)))
    m.attention.set_ctx(ctx)


@pytest.mark.parametrize("M,mode,att", [
    (1, "streamed", dict(max_ctx=200, page_size=32)),
    (2, "streamed", dict(max_ctx=100, page_size=16, kind=tern.TERN_KV_E4M3, window=40, sinks=3)),
    (3, "fused", dict(max_ctx=130, page_size=64)),
    (3, "unfused", dict(max_ctx=130, page_size=64, window=20)),
])
def test_step_attends_over_the_cache(M, mode, att):
    ctx0 = [61, 15, 0][:M]
    m = model(M, mode, **att)
    a = m.attention
    start(m, np.random.default_rng(1), ctx0)
    refs = [{x: getattr(c, x).cpu().numpy().copy() for x in ("k_codes", "k_scales", "v_codes", "v_scales")}
            for c in a.caches]
    table, pages = a.rope.table.cpu().numpy(), a.batch.pages.cpu().numpy()
    kind, rows = att.get("kind", 0), np.arange(M + 1)
    for step in range(3):
        keep = []
        m.step(keep)
        ctx = [c + step + 1 for c in ctx0]
        np.testing.assert_array_equal(a.ctx.cpu().numpy(), ctx)
        pos = np.array([ctx]) - 1
        tag = "attention" if mode == "unfused" else "o_in"
        qkvs = [r[1].cpu().numpy() for r in keep if r[0] == tag]
        outs = [r[-1].cpu().numpy() for r in keep if r[0] == "attention"]
        assert len(qkvs) == len(outs) == LAYERS
        for qkv, out, ref, cache in zip(qkvs, outs, refs, a.caches):
            q, k, v = (qkv[:, i:j].reshape(M, -1, 128) for i, j in ((0, 512), (512, 768), (768, 1024)))
            q_rot, bad = paged.append(q, k, v, pos, table, rows, ctx, pages, ref, kind)
            assert bad == 0
            for x in ("k_codes", "k_scales", "v_codes", "v_scales"):
                np.testing.assert_array_equal(getattr(cache, x).cpu().numpy(), ref[x])
            want = paged.attention(q_rot, rows, ctx, pages, ref, kind, a.window, a.sinks)
            kk, vv, _ = paged.values(np.concatenate([[0], np.cumsum(ctx)]), ctx, pages, ref, kind)
            err = np.abs(out.reshape(M, 4, 128) - want)
            assert np.all(err <= bound(q_rot, kk, vv, 128 ** -0.5, max(ctx)))
    assert int(a.refused) == 0 and tern.tern_device_error() == 0


@pytest.mark.parametrize("M,mode", [(2, "streamed"), (3, "fused")])
def test_graph_decodes_token_after_token(M, mode):
    ctx0 = [30, 7, 12][:M]
    m = model(M, mode, max_ctx=64, page_size=16)
    start(m, np.random.default_rng(2), ctx0)
    for _ in range(4):
        m.step()
    want_x, want_codes = m.x.clone(), [c.k_codes.clone() for c in m.attention.caches]
    graph = m.capture()
    start(m, np.random.default_rng(2), ctx0)
    for _ in range(4):
        graph.replay()
    assert torch.equal(m.x, want_x)
    for c, w in zip(m.attention.caches, want_codes):
        assert torch.equal(c.k_codes, w)
    assert m.attention.ctx.tolist() == [c + 4 for c in ctx0]


def test_tokens_past_the_pages_are_counted():
    m = model(1, "streamed", max_ctx=16, page_size=16)
    start(m, np.random.default_rng(3), [15])
    for _ in range(3):
        m.step()
    assert int(m.attention.refused) == 2 * LAYERS
    assert torch.isfinite(m.x).all()
