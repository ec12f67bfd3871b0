"""The descriptors of the paged calls on the host: the structs whose addresses
a call passes on stay alive until it returns, whatever other threads do to the
descriptors meanwhile.  A stand-in takes the library's place; tensors are the
CPU's."""
import copy
import ctypes
import gc
import pickle
import weakref

import pytest
import torch

from test_abi import _lib


@pytest.fixture
def tern(monkeypatch):
    _lib()
    from ternary_weight_decode_b200 import tern
    monkeypatch.setattr(tern, "_one_device", lambda *t: -1)   # (what get_device says of a CPU tensor)
    monkeypatch.setattr(tern, "_call_stream", lambda dev, stream: 0)
    return tern


def descriptors(tern):
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)
    plan = tern.RopePlan(torch.zeros(8, 64, 2), [30, 34])
    cache = tern.PagedCache.empty(tern.TERN_KV_INT8, 2, 128, 32, 3, device="cpu")
    batch = tern.PagedBatch(i32(0, 1, 3), i32(5, 9), i32(0, -1, 2, 1).view(2, 2), 3, 2, 40)
    return plan, cache, batch


class Library:
    """Every entry point: the descriptors' structs are made anew, as by another thread, and those that
    the call was given have to be alive still."""

    def __init__(self, tern, monkeypatch, described):
        self.alive, self.calls = {}, []
        for cls in (tern.RopePlan, tern.PagedCache, tern.PagedBatch):
            monkeypatch.setattr(cls, "struct", self.watched(cls.struct))

        def entry(name):
            def call(*args):
                for d in described:
                    d.__dict__.pop("_kept", None)
                    d.described()
                gc.collect()
                self.calls.append(name)
                for a in args:
                    if a in self.alive:
                        assert self.alive[a]() is not None, name
                return 0
            return call
        for name in ("tern_rope", "tern_kv_append_paged", "tern_kv_read_paged", "tern_attention_paged",
                     "tern_attention_paged_workspace_bytes"):
            setattr(self, name, entry(name))

    def watched(self, struct):
        def made(d):
            s = struct(d)
            self.alive[ctypes.addressof(s)] = weakref.ref(s)
            return s
        return made


def test_structs_live_until_the_call_returns(tern, monkeypatch):
    plan, cache, batch = descriptors(tern)
    L = Library(tern, monkeypatch, (plan, cache, batch))
    monkeypatch.setattr(tern, "_lib", L)
    q, k, v = torch.zeros(3, 4, 128), torch.zeros(3, 2, 128), torch.zeros(3, 2, 128)
    pos, ws = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(4096)
    out = torch.zeros_like(q)
    tern.tern_rope(plan, pos, q, out)
    tern.tern_kv_append_paged(q, k, v, pos, plan, batch, cache, q)
    tern.tern_kv_read_paged(batch, cache, k, v)
    tern.tern_attention_paged(q, batch, cache, out, ws)
    tern.tern_attention_paged_workspace_bytes(4, cache)
    assert len(L.calls) == 5


def test_a_call_takes_its_sizes_from_the_struct_it_passes(tern, monkeypatch):
    """A row count that another thread sets while a call checks its tensors does not split the two."""
    plan, cache, batch = descriptors(tern)
    seen = []

    class L:
        @staticmethod
        def tern_attention_paged(q, ldq, Hq, b, c, *rest):
            seen.append((tern.tern_paged_batch.from_address(b).T, tern.tern_paged_cache.from_address(c).Hkv))
            return 0
    monkeypatch.setattr(tern, "_lib", L)
    heads = tern._heads

    def interrupted(t, dev, T, H, D):
        batch.T = 99
        return heads(t, dev, T, H, D)
    monkeypatch.setattr(tern, "_heads", interrupted)
    q = torch.zeros(3, 4, 128)
    tern.tern_attention_paged(q, batch, cache, torch.zeros_like(q), torch.zeros(4096))
    assert seen == [(3, 2)]


@pytest.mark.parametrize("name", ["k_codes", "k_scales", "v_codes", "v_scales"])
def test_a_cache_tensor_resized_in_place_is_refused(tern, name):
    _, cache, _ = descriptors(tern)
    cache.described()
    t = getattr(cache, name)
    at = t.data_ptr()
    t.resize_(2, *t.shape[1:])
    assert t.data_ptr() == at
    with pytest.raises(AssertionError):
        cache.described()


@pytest.mark.parametrize("name", ["row_start", "ctx", "pages"])
def test_a_batch_tensor_resized_in_place_is_refused(tern, name):
    _, _, batch = descriptors(tern)
    batch.described()
    t = getattr(batch, name)
    at = t.data_ptr()
    t.resize_(1, *t.shape[1:])
    assert t.data_ptr() == at
    with pytest.raises(AssertionError):
        batch.described()


def test_tensors_resized_together_are_followed(tern):
    plan, cache, batch = descriptors(tern)
    for d in (plan, cache, batch):
        d.described()
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.resize_(2, *t.shape[1:])
    batch.row_start.resize_(2), batch.ctx.resize_(1), batch.pages.resize_(1, 2)
    plan.table.resize_(8, 32, 2)
    plan.sections[:] = [20, 12]
    assert cache.described()[3].n_pages == 2
    assert (batch.described()[3].B, batch.described()[3].pages_ld) == (1, 2)
    assert plan.described()[3].rot_dim == 64
    plan.table.resize_(4, 64, 2)   # the same number of elements
    assert (plan.described()[3].n_pos, plan.described()[3].rot_dim) == (4, 128)


@pytest.mark.parametrize("copied", [copy.copy, copy.deepcopy, lambda d: pickle.loads(pickle.dumps(d))])
def test_descriptors_that_were_used_are_copied(tern, copied):
    for d in descriptors(tern):
        address, _, _, kept = d.described()
        other = copied(d)
        assert type(other) is type(d) and "_kept" not in other.__dict__
        assert other.described()[0] != address and d.described()[3] is kept
        for name, t in other.__dict__.items():
            if isinstance(t, torch.Tensor):
                assert torch.equal(t, getattr(d, name))
