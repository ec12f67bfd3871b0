"""Pins of the numpy forms of the rotary embedding and the paged 8-bit cache."""
import numpy as np
import pytest

from oracle import paged


def test_rotation_is_a_rotation_and_its_inverse_undoes_it():
    rng = np.random.default_rng(0)
    table = paged.rope_table(10000.0, 64, 500)
    pos = rng.integers(0, 500, (3, 9))
    x = rng.standard_normal((9, 2, 80)).astype(np.float32)
    for inter in (False, True):
        y, bad = paged.rope(x, pos, table, [8, 12, 12], inter)
        assert bad == 0
        np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-6)
        np.testing.assert_array_equal(y[..., 64:], x[..., 64:])
        z, _ = paged.rope(y, pos, table, [8, 12, 12], inter, inverse=True)
        np.testing.assert_allclose(z, x, atol=2e-6)
    # equal positions on every axis: the product of a query and a key depends on their distance alone
    q, k = x[:1, :1, :64], x[1:2, :1, :64]
    dots = [float((paged.rope(q, np.full((3, 1), p + 7), table, [8, 12, 12])[0]
                   * paged.rope(k, np.full((3, 1), p), table, [8, 12, 12])[0]).sum()) for p in (0, 100, 400)]
    assert max(dots) - min(dots) < 1e-4


def test_e4m3_codes_match_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(1)
    y = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.uniform(-4, 2.5, 4000),
                        paged._E4M3[np.isfinite(paged._E4M3)], [448.0, 464.0, -460.0, 2.0 ** -10, 3 * 2.0 ** -11]])
    y = np.clip(y, -448, 448).astype(np.float32)
    ref = torch.from_numpy(y).to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(paged.to_codes(y, paged.E4M3), ref.view(torch.uint8).numpy())
    np.testing.assert_array_equal(paged.from_codes(paged.to_codes(y, paged.E4M3), paged.E4M3), ref.float().numpy())


@pytest.mark.parametrize("kind,top", [(paged.INT8, 127.0), (paged.E4M3, 448.0)])
def test_scale_is_the_least_power_of_two(kind, top):
    for a in (1e-3, 1.0, top, top * 1.0001, 3.7, 0.999 * top / 4):
        s = float(paged.pow2_scale(a, kind))
        assert a <= top * s and a > top * s / 2 and np.log2(s) == round(np.log2(s))
    assert float(paged.pow2_scale(0.0, kind)) == 2.0 ** -100


@pytest.mark.parametrize("kind", [paged.INT8, paged.E4M3])
def test_append_in_portions_stays_within_a_step(kind):
    """Tokens one by one, growing in size: the error of an int8 value is at
    most one step of the final scale (half a step when written, and at most
    half the later scale for each doubling), of an e4m3 value half a unit of
    its last place, or of the smallest subnormal under the final scale."""
    rng = np.random.default_rng(2)
    cache = {"k_codes": np.zeros((2, 1, 32, 8), np.uint8), "v_codes": np.zeros((2, 1, 32, 8), np.uint8),
             "k_scales": np.zeros((2, 1, 2), np.float32), "v_scales": np.zeros((2, 1, 2), np.float32)}
    table = paged.rope_table(100.0, 8, 4)
    pages = np.array([[1]])
    x = (rng.standard_normal((20, 1, 8)) * 1.5 ** np.arange(20)[:, None, None]).astype(np.float32)
    for t in range(20):
        paged.append(x[t:t + 1], x[t:t + 1], x[t:t + 1], np.zeros((1, 1), int), table, [0, 1], [t + 1], pages, cache,
                     kind)
    _, v, bad = paged.values([0, 20], [20], pages, cache, kind)
    assert bad == 0
    s = cache["v_scales"][1, 0][np.arange(20) // 16][:, None, None]
    bound = s if kind == paged.INT8 else np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -9)
    assert np.all(np.abs(v - x) <= bound)


def test_attention_closed_forms():
    """Equal keys: the mean of the visible values; a far larger key: its value."""
    cache = {"k_codes": np.full((3, 1, 16, 128), 1, np.uint8), "v_codes": np.zeros((3, 1, 16, 128), np.uint8),
             "k_scales": np.ones((3, 1, 1), np.float32), "v_scales": np.full((3, 1, 1), 0.5, np.float32)}
    for p in range(3):
        cache["v_codes"][p, 0] = (16 * p + np.arange(16))[:, None]
    pages = np.array([[0, 1, 2]])
    q = np.ones((2, 2, 128), np.float32)
    o = paged.attention(q, [0, 2], [40], pages, cache, 0)
    np.testing.assert_allclose(o[:, :, 0], [[38 / 2 * 0.5] * 2, [39 / 2 * 0.5] * 2])
    o = paged.attention(q, [0, 2], [40], pages, cache, 0, window=5, sinks=2)
    seen = np.array([0, 1, 35, 36, 37, 38, 39])
    np.testing.assert_allclose(o[1, 0, 0], seen.mean() * 0.5)
    o = paged.attention(q, [0, 2], [40], np.array([[0, -1, 2]]), cache, 0)
    np.testing.assert_allclose(o[1, 0, 0], np.r_[0:16, 32:40].mean() * 0.5)
    assert np.all(paged.attention(q, [0, 2], [40], np.array([[-1, 3, -1]]), cache, 0) == 0)
