"""Plain 64-bit forms of the e4m3 and grouped products, with the error bounds
the GPU tests use.  Written from the definitions, apart from the library's
code.

Error of a product (products are exact: e4m3 x e4m3 has 8 significant bits,
bf16 x bf16 16, f16 x f16 22, all within f32's 24).  The tensor core adds the
products of one instruction (32 bytes of K: 32 e4m3 or 16 16-bit values) and
the running f32 sum; an f32 addition that may truncate is off by at most 2^-23
of the larger magnitude, so n terms in one instruction and i instructions in a
row are off by at most (n + i) 2^-23 S, S the sum of the terms' magnitudes.
e4m3: n = 32, i = 4 per block of 128; the scale product rounds once (2^-24) and
each block's fma once (2^-24):  (36 * 2 + 1 + blocks) 2^-24 S.
16-bit: n = 16, i = ceil(K/16):  (16 + ceil(K/16)) 2^-23 S.
Rounding y to its type adds half a step, eps/2 |y|, and half of the smallest
subnormal (f16: 2^-25).
A split K range adds at most 8 parts in f32: 8 * 2^-24 S more.
"""
import numpy as np

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}


def e4m3_table():
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        a = np.nan if (e == 15 and m == 7) else \
            m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = -a if s else a
    return v


TABLE = e4m3_table()


def e4m3_codes(v):
    """Code of the nearest e4m3 value (ties to the even code, saturating);
    non-finite values give the NaN code 0x7F."""
    v = np.asarray(v, np.float64)
    pos = TABLE[:127]
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(a >= 448.0, 126, c)
    c = c | np.where(np.signbit(v), 0x80, 0)
    return np.where(np.isfinite(v), c, 0x7F).astype(np.uint8)


def block_scale(top):
    """The smallest 2^k, k >= -126, with top <= 448 * 2^k (1 for top = 0)."""
    top = np.asarray(top, np.float64)
    k = np.full(top.shape, -126)
    for i in range(-126, 121):
        k = np.where(top > 448.0 * 2.0 ** i, i + 1, k)
    return np.where(top > 0, 2.0 ** k.astype(np.float64), 1.0)


def quantize(x):
    """(codes, scales) of rows x (any float array, taken as 64-bit values)."""
    x = np.asarray(x, np.float64)
    n, k = x.shape
    nb = -(-k // 128)
    q = np.empty((n, k), np.uint8)
    s = np.empty((n, nb))
    for b in range(nb):
        blk = x[:, b * 128:(b + 1) * 128]
        s[:, b] = block_scale(np.where(np.isfinite(blk), np.abs(blk), 0.0).max(1))
        q[:, b * 128:(b + 1) * 128] = e4m3_codes(blk / s[:, b:b + 1])
    return q, s


def row_values(q, s):
    return TABLE[q] * np.repeat(s, 128, axis=1)[:, :q.shape[1]]


def matrix_values(q, s):
    n, k = q.shape
    return TABLE[q] * np.repeat(np.repeat(s, 128, axis=0)[:n], 128, axis=1)[:, :k]


def product(x, w, terms):
    """(y, error bound before rounding) of x w^T; `terms` of 2^-24 S."""
    y = x @ w.T
    return y, terms * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T)


def f8_terms(k):
    return 36 * 2 + 1 + -(-k // 128) + 8


def wide_terms(k):
    return 2 * (16 + -(-k // 16)) + 8


def rounded(y, err, kind):
    """Tolerance of y after rounding to `kind`."""
    return err + HALF_STEP[kind] * (np.abs(y) + err) + TINY[kind]
