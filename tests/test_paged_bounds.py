"""The bounds that the paged attention is held to, on the host with numpy forms of
its arithmetic: the whole of it keeps them, with a digit less it does not."""
import numpy as np
import pytest

from paged_bounds import (E4M3, INT8, RMS_FACTOR, border_query, bound_row, fp32_row, query_digits, rms, row_by_digits,
                          softmax_row)
from oracle import paged

D = 128


def tokens(rng, n, kind):
    """Keys and values of n tokens as the append would hold normal ones."""
    out = []
    for _ in range(2):
        x = rng.standard_normal((n, D)) * (rng.random((-(-n // 16), 1, 1)) + 0.25).repeat(16, 1).reshape(-1, 1)[:n]
        s = np.array([paged.pow2_scale(float(np.abs(x[i:i + 16]).max()), kind) for i in range(0, n, 16)], np.float64)
        s = s.repeat(16)[:n]
        out += [paged.from_codes(paged.to_codes((x / s[:, None]).astype(np.float32), kind), kind) * s[:, None], s]
    return out[0], out[2], out[3]


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("n", [1, 33, 333, 5000])
def test_the_bound_holds_for_the_digits(n, kind):
    rng = np.random.default_rng(n)
    for _ in range(4):
        q = (rng.standard_normal(D) * 1.5).astype(np.float32)
        K, V, s = tokens(rng, n, kind)
        tol = bound_row(q, K, V, s, D ** -0.5, kind)
        err = np.abs(row_by_digits(q, K, V, s, D ** -0.5, kind) - softmax_row(q, K, V, D ** -0.5)[2])
        assert np.all(err <= tol)


@pytest.mark.parametrize("kind,drop_q,drop_w", [(INT8, 1, 0), (INT8, 0, 1), (E4M3, 2, 0), (E4M3, 0, 2)])
@pytest.mark.parametrize("n", [33, 333, 5000])
@pytest.mark.parametrize("spread", [1.5, 6.0])
def test_the_mean_error_sees_a_lost_digit(n, spread, kind, drop_q, drop_w):
    """Against that of the plain fp32 form: with all digits it passes by far, of int8 a single one left out fails, of
    e4m3 (where the last of the five is of an fp32 rounding's size) two."""
    rng = np.random.default_rng(n)
    errors = {"plain": [], "whole": [], "less": []}
    for _ in range(6):
        q = (rng.standard_normal(D) * spread).astype(np.float32)
        K, V, s = tokens(rng, n, kind)
        out = softmax_row(q, K, V, D ** -0.5)[2]
        errors["plain"].append(fp32_row(q, K, V, D ** -0.5) - out)
        errors["whole"].append(row_by_digits(q, K, V, s, D ** -0.5, kind) - out)
        errors["less"].append(row_by_digits(q, K, V, s, D ** -0.5, kind, drop_q, drop_w) - out)
    plain, whole, less = (rms(errors[k]) for k in ("plain", "whole", "less"))
    assert whole <= RMS_FACTOR / 4 * plain and less > RMS_FACTOR * plain, (plain, whole, less)


def test_query_digits():
    rng = np.random.default_rng(0)
    for top in (1.0, 1.98, 1.99, 2.0, 3.97, 0.7):
        q = rng.uniform(-top, top, 1000).astype(np.float32)
        q[0] = -top
        assert np.abs(query_digits(q, INT8) - q).max() <= 2.0 ** -22.9 * np.abs(q).max()
        e = np.abs(query_digits(q, E4M3) - q)
        assert np.all(e <= np.maximum(2.0 ** -20 * np.abs(q), 2.0 ** -32 * np.abs(q).max()))


def test_the_border_query_tells_2_to_the_minus_22_from_half_of_it():
    rng = np.random.default_rng(3)
    q, signs = border_query(rng)
    assert np.all(np.abs(query_digits(q, INT8) - q) <= 2.0 ** -22.9)
    V, s = np.concatenate([np.full((1, D), 100.0), np.full((1, D), -100.0)]), np.ones(2)
    K = 100.0 * np.stack([signs, -signs])
    tol = bound_row(q, K, V, s, D ** -0.5, INT8)
    out = softmax_row(q, K, V, D ** -0.5)[2]
    assert np.all(np.abs(row_by_digits(q, K, V, s, D ** -0.5, INT8) - out) <= tol)
    coarse = np.rint(q.astype(np.float64) * 2 ** 21) / 2 ** 21
    assert np.all(np.abs(softmax_row(coarse, K, V, D ** -0.5)[2] - out) > tol)
