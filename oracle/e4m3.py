"""The e4m3 block format in numpy: test infrastructure, no code shared with the GPU path.

Codes are uint8 bit patterns; a code's value comes from a table built from the
format's definition (sign, 4 exponent bits with bias 7, 3 mantissa bits; 0x7f and
0xff NaN), rounding from a search among the table's values.
"""

import numpy as np

BLOCK = 128


def _table():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = np.nan if (e, m) == (15, 7) else (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[c] = -a if c & 0x80 else a
    return v


VALUE = _table()
_POS = VALUE[:127]  # ascending: codes 0 .. 126
_MID = (_POS[1:] + _POS[:-1]) / 2  # exact in f64


def decode(codes):
    return VALUE[np.asarray(codes, np.uint8)]


def round_codes(t):
    """f64 -> codes, nearest, ties to the even code, saturating, NaN to NaN."""
    t = np.asarray(t, np.float64)
    a = np.abs(t)
    lo = np.searchsorted(_MID, a, side="left")   # midpoints below a
    hi = np.searchsorted(_MID, a, side="right")  # and those equal to it
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi)).astype(np.uint8)
    code = np.where(np.isnan(t), 0x7F, code)
    return (code | (np.signbit(t).astype(np.uint8) << 7)).astype(np.uint8)


def blocks(n):
    return -(-n // BLOCK)


def block_top(v):
    """max(max|v|, 2^-100) of every block of the rows of v; NaN passed over."""
    rows, k = v.shape
    p = np.zeros((rows, blocks(k) * BLOCK), v.dtype)
    p[:, :k] = np.where(np.isnan(v), 0, np.abs(v))
    return np.maximum(p.reshape(rows, -1, BLOCK).max(axis=2), v.dtype.type(2.0 ** -100))


def spread(d, k):
    """One value per block -> one per column."""
    return np.repeat(d, BLOCK, axis=1)[:, :k]


def quantize(v):
    """f32 [rows, k] -> (codes, f32 scales), the two roundings to f32 as defined."""
    v = np.ascontiguousarray(v, np.float32)
    a = block_top(v)
    with np.errstate(all="ignore"):
        t = (v * spread(np.float32(448) / a, v.shape[1])).astype(np.float32)
        return round_codes(t), a / np.float32(448)


def norm(s, gamma, eps):
    """f32 rows s -> the f32 rows (s * r) * gamma."""
    s = np.asarray(s, np.float32)
    r = (1.0 / np.sqrt(np.mean(s.astype(np.float64) ** 2, axis=1, keepdims=True) + np.float64(np.float32(eps))))
    return (s * r.astype(np.float32)) * np.asarray(gamma, np.float32)


def product(wq, wd, xq, xd):
    """(y, sum of |terms|) in f64: y[m][n] = sum_b xd wd S_b."""
    w = decode(wq) * np.repeat(np.repeat(wd.astype(np.float64), BLOCK, axis=0)[: wq.shape[0]], BLOCK, axis=1)[:, : wq.shape[1]]
    x = decode(xq) * spread(xd.astype(np.float64), xq.shape[1])
    return x @ w.T, np.abs(x) @ np.abs(w).T


def weight(rng, n, k, scale=0.02):
    """Random normal weights as (codes, scales)."""
    w = np.zeros((blocks(n) * BLOCK, blocks(k) * BLOCK))
    w[:n, :k] = rng.standard_normal((n, k)) * scale
    t = w.reshape(blocks(n), BLOCK, blocks(k), BLOCK)
    a = np.maximum(np.abs(t).max(axis=(1, 3)), 2.0 ** -100)
    q = round_codes(t * (448.0 / a)[:, None, :, None]).reshape(w.shape)
    return np.ascontiguousarray(q[:n, :k]), (a / 448.0).astype(np.float32)
