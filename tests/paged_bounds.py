"""Bounds of the paged attention's error, row by row, counted from what
include/tern.h promises of its arithmetic; and numpy forms of that arithmetic
(queries and softmax weights as digits), whole or with a digit left out."""
import numpy as np

INT8, E4M3 = 0, 1
LOG2E = 1.4426950408889634


def exponent(s):
    """The least integer e with s <= 2^e."""
    return np.ceil(np.log2(s))


def softmax_row(q, K, V, scale):
    """(scores in log2, weights, output) in 64 bits."""
    x = K @ q.astype(np.float64) * (scale * LOG2E)
    p = np.exp2(x - x.max())
    p /= p.sum()
    return x, p, p @ V


def bound_row(q, K, V, v_scales, scale, kind, tiles=None):
    """The largest error [D] of one row and head over its visible tokens: K, V [n, D] their values, v_scales [n]
    their value scales.  A relative change eps_j of weight j moves the output by at most sum_j p_j eps_j |v_j - out|.
    tiles [n]: the product that the reference of each token's weight follows (the largest of all by default)."""
    x, p, out = softmax_row(q, K, V, scale)
    n = len(x)
    q = np.abs(q.astype(np.float64))
    if kind == INT8:   # a query is held to 2^-22.9 of its row's largest element, and the products are exact
        dx = 2.0 ** -22.9 * q.max() * np.abs(K).sum(1)
    else:              # to 2^-20 of each element; the sums of a tile's 128 products add four times in fp32
        dx = (2.0 ** -20 + 16 * 2.0 ** -24) * (np.abs(K) @ q)
    dx = dx * abs(scale) * LOG2E
    # the constants and the products that make a score; the value scale's exponent added, the reference taken off
    dx = dx + (8 * np.abs(x) + (x.max() - x) + 64) * 2.0 ** -24
    # 2^-22 of the exponential and the roundings behind it; the digits of e4m3
    eps = np.log(2.0) * dx + 2.0 ** -21 + (2.0 ** -20 if kind == E4M3 else 0.0)
    e = exponent(v_scales)
    T = p * np.exp2(e)
    ref = np.full(n, T.max()) if tiles is None else tiles
    quantum = ref * 2.0 ** (-27 if kind == INT8 else -28)
    lost = (quantum[:, None] * np.abs(V) / np.exp2(e)[:, None]).sum(0)
    # sums: int8 exact up to the joining of chains; e4m3's add in fp32 inside a chain of 16 tiles, four times a tile
    steps = 16 + n / 4096 if kind == INT8 else 128 + n / 2048
    sums = steps * 2.0 ** -24 * (p @ np.abs(V)) + (16 + n / 256) * 2.0 ** -24 * np.abs(out)
    return (p * eps) @ np.abs(V - out) + lost + sums


# The root mean square of the kernel's errors is held to this times that of the plain fp32 form on the same inputs: its
# exponential is off by four half steps where the plain one's is by one, and the tensor cores' sums by two where plain ones
# are by one; what the digits leave out is of an fp32 rounding's size.
RMS_FACTOR = 8.0


def fp32_row(q, K, V, scale):
    """The plain form in fp32."""
    K, V = K.astype(np.float32), V.astype(np.float32)
    x = (K @ q.astype(np.float32)) * np.float32(scale)
    w = np.exp(x - x.max())
    return (w @ V) / w.sum()


def rms(errors):
    return float(np.sqrt(np.mean(np.square(np.asarray(errors, np.float64)))))


def query_digits(q, kind, drop=0):
    """A query as its digits hold it, without the `drop` lowest."""
    q = q.astype(np.float64)
    m = np.abs(q).max()
    if m == 0:
        return q
    if kind == INT8:
        e = 22 - np.floor(np.log2(m))
        if m * 2.0 ** e > 1.984375 * 2.0 ** 22:
            e -= 1
        n = np.rint(q * 2.0 ** e)
        return np.rint(n / 256 ** drop) * 256 ** drop / 2.0 ** e   # (signed digits: leaving them out rounds)
    e = 7 - np.floor(np.log2(m))
    return e4m3_digits(q * 2.0 ** e, 5 - drop) / 2.0 ** e


def e4m3_digits(x, count):
    """x as `count` e4m3 digits, each the nearest to what is left, a 16th as large."""
    out, left, unit = np.zeros_like(x), x.copy(), 1.0
    for _ in range(count):
        a = np.maximum(np.abs(left), 2.0 ** -40)
        step = np.exp2(np.maximum(np.floor(np.log2(a)), -6) - 3)
        d = np.rint(left / step) * step
        out += d * unit
        left = (left - d) * 16
        unit /= 16
    return out


def row_by_digits(q, K, V, v_scales, scale, kind, drop_q=0, drop_w=0):
    """The output of one row whose query and weights are held as digits (one reference for all tokens)."""
    x = K @ query_digits(q, kind, drop_q) * (scale * LOG2E)
    w = np.exp2(x - x.max())
    prod = w * v_scales
    c = exponent(prod.max()) + 6
    if kind == INT8:
        u = np.rint(prod * np.exp2(32 - c))
        u = np.floor(u / 256 ** drop_w) * 256 ** drop_w / np.exp2(32 - c)
    else:
        u = e4m3_digits(prod * np.exp2(8 - c), 5 - drop_w) / np.exp2(8 - c)
    return (u @ (V / v_scales[:, None])) / w.sum()


def border_query(rng):
    """(q, signs) [D = 128]: a query whose largest element is just 1 and whose others lie half-way between multiples of
    2^-21; kept to those multiples, all errors would have the signs given, while q . signs is about 0."""
    m = rng.integers(1 << 17, 1 << 20, 64) * 2
    m = np.concatenate([m + 1, m])             # odd ones round up, even ones down
    q = ((2 * m + 1) * 2.0 ** -22).astype(np.float32)
    q[63], q[127] = 1.0, 1.0 - 2.0 ** -21
    return q, np.concatenate([np.ones(64), -np.ones(64)])
