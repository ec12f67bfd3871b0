"""The paged attention whose waits run out: with a budget shorter than they
ordinarily take, a call records the device error and ends, whichever wait it
was, writes nothing but its rows, and leaves the context usable."""
import numpy as np
import pytest
import torch

from test_gpu_paged import E4M3, INT8
from test_gpu_paged_edges import Call
from ternary_weight_decode_b200 import tern

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,ctx,kind,Hq,Hkv,window", [([1] * 3, [9000, 40, 3000], INT8, 10, 2, 0),   # 8 rows an item
                                                      ([1] * 3, [9000, 40, 3000], E4M3, 10, 2, 0),
                                                      ([3, 1], [5000, 700], INT8, 10, 2, 300),       # 16
                                                      ([30, 200], [900, 3100], E4M3, 4, 2, 0),
                                                      ([30, 200], [900, 3100], INT8, 4, 2, 0)])      # 32
def test_a_wait_that_runs_out_ends_the_call(n, ctx, kind, Hq, Hkv, window):
    c = Call(3, n, ctx, kind, Hq, Hkv, window=window)
    c.window = window
    T, pad = sum(n), 5
    wide = torch.full((T + pad, Hq, 128), -2.0, device="cuda")
    c.out = wide[:T]
    ws = tern.attention_paged_workspace(Hq, c.dev)
    guard = torch.full((ws.numel() + 4096,), 7.0, device="cuda")
    ws = guard[:ws.numel()]
    before = [getattr(c.dev, x).clone() for x in ("k_codes", "k_scales", "v_codes", "v_scales")]
    ran_out = 0
    assert tern.tern_device_error() == 0
    try:
        for budget in (1, 300, 1000, 3000, 10000, 30000):
            ws.zero_()
            tern.tern_debug_paged_wait_budget(budget)
            c.run(ws)
            code = tern.tern_device_error()
            assert code in (0, 1)
            ran_out += code
            if code == 0:
                c.check()
            assert torch.all(wide[T:] == -2.0) and torch.all(guard[ws.numel():] == 7.0)
    finally:
        tern.tern_debug_paged_wait_budget(0)
    assert ran_out > 0
    for x, was in zip(("k_codes", "k_scales", "v_codes", "v_scales"), before):
        assert torch.equal(getattr(c.dev, x).view(torch.uint8), was.view(torch.uint8))
    ws.zero_()
    c.run(ws)
    c.check()
    assert tern.tern_device_error() == 0 and not ws[:1024].view(torch.int32).any()
