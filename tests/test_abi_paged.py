"""Host checks of the rotary embedding and the paged cache: bad arguments are
refused before any launch (no GPU is needed to see the refusal)."""
import ctypes

import pytest

from test_abi import _lib

P = 4096  # a 16-byte aligned address that no refused call reads


def _structs(rope=None, batch=None, cache=None):
    from ternary_weight_decode_b200 import tern
    r = dict(table=P, n_pos=10, rot_dim=128, axes=1, section=(64, 0, 0), flags=0, reserved=0)
    b = dict(B=2, T=4, max_rows=3, max_ctx=40, row_start=P, ctx=P, pages=P, pages_ld=2, reserved=0)
    c = dict(kind=0, Hkv=2, D=128, page_size=32, n_pages=6, reserved=0, k_codes=P, k_scales=P, v_codes=P, v_scales=P)
    r.update(rope or {}), b.update(batch or {}), c.update(cache or {})
    r["section"] = (ctypes.c_int32 * 3)(*r["section"])
    return tern.tern_rope_plan(**r), tern.tern_paged_batch(**b), tern.tern_paged_cache(**c)


def _append(rope=None, batch=None, cache=None, q=P, ldq=512, Hq=4, k=P, ldk=256, v=P, ldv=256, pos=P, out=P, ldo=512,
            bad=None):
    L = _lib()
    r, b, c = _structs(rope, batch, cache)
    st = L.tern_kv_append_paged(q, ldq, Hq, k, ldk, v, ldv, pos, ctypes.addressof(r), ctypes.addressof(b),
                                ctypes.addressof(c), out, ldo, bad, None)
    return st, L.tern_last_error()


def _attend(batch=None, cache=None, q=P, ldq=512, Hq=4, window=0, sinks=0, scale=0.1, out=2 * P, ldo=512, ws=P,
            nbytes=1 << 30):
    L = _lib()
    _, b, c = _structs(None, batch, cache)
    st = L.tern_attention_paged(q, ldq, Hq, ctypes.addressof(b), ctypes.addressof(c), window, sinks, scale, out, ldo,
                                ws, nbytes, None)
    return st, L.tern_last_error()


BAD_CACHE = [dict(kind=2), dict(Hkv=0), dict(page_size=8), dict(page_size=24), dict(page_size=8192), dict(n_pages=0),
             dict(reserved=1), dict(k_codes=P + 8), dict(v_codes=None), dict(k_scales=P + 2), dict(v_scales=None)]
BAD_BATCH = [dict(B=0), dict(B=4097), dict(T=-1), dict(max_rows=0), dict(max_ctx=0), dict(pages_ld=0),
             dict(row_start=None), dict(ctx=P + 2), dict(pages=None), dict(reserved=1)]


@pytest.mark.parametrize("kw", BAD_CACHE)
def test_bad_caches(kw):
    assert _append(cache=kw)[0] == 1
    assert _attend(cache=kw)[0] == 1


@pytest.mark.parametrize("kw", BAD_BATCH)
def test_bad_batches(kw):
    st, msg = _append(batch=kw)
    assert st == 1 and b"tern_kv_append_paged" in msg
    st, msg = _attend(batch=kw)
    assert st == 1 and b"tern_attention_paged" in msg


def test_what_this_build_does_not_take():
    assert _append(cache=dict(D=64), rope=dict(rot_dim=64, section=(32, 0, 0)))[0] == 3
    assert _attend(cache=dict(D=256))[0] == 3
    assert _attend(cache=dict(n_pages=1 << 25))[0] == 3


@pytest.mark.parametrize("kw", [dict(rot_dim=12), dict(rot_dim=136), dict(rot_dim=0), dict(axes=0), dict(axes=4),
                                dict(section=(60, 0, 0)), dict(section=(0, 64, 0)), dict(section=(65, -1, 0), axes=2),
                                dict(flags=4), dict(reserved=1), dict(n_pos=0), dict(table=P + 8), dict(table=None)])
def test_bad_rotary_plans(kw):
    L = _lib()
    assert _append(rope=kw)[0] == 1
    r, _, _ = _structs(kw)
    assert L.tern_rope(ctypes.addressof(r), P, 3, 2, 128, P, 256, P, 256, None, None) == 1
    assert b"tern_rope" in L.tern_last_error()


@pytest.mark.parametrize("kw", [dict(q=P + 4), dict(ldq=510), dict(ldq=508), dict(Hq=0), dict(k=None), dict(ldk=252),
                                dict(v=P + 8), dict(ldv=258), dict(pos=None), dict(pos=P + 1), dict(out=None),
                                dict(ldo=516), dict(bad=P + 2)])
def test_bad_append_rows(kw):
    assert _append(**kw)[0] == 1


@pytest.mark.parametrize("kw", [dict(Hq=3), dict(Hq=0), dict(q=None), dict(out=P), dict(out=2 * P + 4), dict(ldo=500),
                                dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf")),
                                dict(ws=None), dict(ws=P + 8)])
def test_bad_attention_calls(kw):
    assert _attend(**kw)[0] == 1


def test_no_rows_is_a_call_that_does_nothing():
    L = _lib()
    assert _append(batch=dict(T=0), q=None, k=None, v=None, pos=None, out=None)[0] == 0
    assert _attend(batch=dict(T=0), q=None, out=None, ws=None)[0] == 0
    r, b, c = _structs(None, dict(T=0))
    assert L.tern_kv_read_paged(ctypes.addressof(b), ctypes.addressof(c), None, 0, None, 0, None, None) == 0
    assert L.tern_rope(ctypes.addressof(r), None, 0, 2, 128, None, 0, None, 0, None, None) == 0


@pytest.mark.parametrize("args", [(0.0, 1.0, 64, 10, P), (1e4, -1.0, 64, 10, P), (float("nan"), 1.0, 64, 10, P),
                                  (float("inf"), 1.0, 64, 10, P), (1e4, 1.0, 60, 10, P), (1e4, 1.0, 64, 0, P),
                                  (1e4, 1.0, 64, 10, P + 8), (1e4, 1.0, 64, 10, None)])
def test_bad_tables(args):
    assert _lib().tern_rope_table(*args, None) == 1


@pytest.mark.parametrize("T,H,D,ldx,ldy,y", [(-1, 2, 128, 256, 256, P), (3, 0, 128, 256, 256, P),
                                             (3, 2, 132, 264, 264, P), (3, 2, 520, 1040, 1040, P),
                                             (3, 2, 128, 252, 256, P), (3, 2, 128, 258, 256, 2 * P),
                                             (3, 2, 128, 256, 260, P), (3, 2, 128, 256, 256, P + 4)])
def test_bad_rope_rows(T, H, D, ldx, ldy, y):
    L = _lib()
    r, _, _ = _structs()
    assert L.tern_rope(ctypes.addressof(r), P, T, H, D, P, ldx, y, ldy, None, None) == 1


def test_read_refuses_bad_rows():
    L = _lib()
    _, b, c = _structs()
    for args in ((None, 256, P, 256), (P, 252, P, 256), (P, 256, P + 4, 256), (P, 256, P, 258)):
        assert L.tern_kv_read_paged(ctypes.addressof(b), ctypes.addressof(c), *args, None, None) == 1


def test_workspace_query_refuses():
    L = _lib()
    _, _, c = _structs()
    n = ctypes.c_size_t()
    assert L.tern_attention_paged_workspace_bytes(3, ctypes.addressof(c), ctypes.byref(n)) == 1
    assert L.tern_attention_paged_workspace_bytes(4, ctypes.addressof(c), None) == 1
    assert L.tern_attention_paged_workspace_bytes(4, None, ctypes.byref(n)) == 1
