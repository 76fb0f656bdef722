"""Plain 64-bit forms of the steps around an MoE layer's products and of the
products with 4-bit weights, with the error bounds the GPU tests use.  Written
from the definitions, apart from the library's code.

u = 2^-24, half a step of f32: one f32 operation is off by at most u of its result.

Routing weights, w = exp(l - top) / z.  The argument l - top is off by u |l - top|,
which the exponential turns into as much relative error; expf itself is off by at
most one ulp, 2 u.  z adds at most 32 values in a lane and 5 more over the warp, all
positive: 37 u, and each of its terms is off as the numerator is.  The division
adds u.  With D the largest l - top of a term that is not 0 in f32 (at most 104):
  (2 (2 + D) + 37 + 1) u of w, and a few subnormal steps, 2^-146.
Gradient of the logits.  c = sum w dw over up to 16 slots: a product and 5 sums, 6 u C
with C = sum |w dw|; dw - c and its factors round once each, and the two terms of
an expert named twice add u.  Renormalised: u |w| (8 C + 4 (|dw| + |c|)).  Else p, formed
as above and by a reciprocal and a product (2 u more): its error times |g - c|, and
u p (8 C + 4 (|g| + |c|)), g up to 16 slots' dw: 16 u p |g| more.
Weighted sum: k fused products and sums and the residual, (k + 1) u (sum |w y| + |r|).
Gradient of a weight: products and sums of `cols` values, by threads that add at
most ceil(cols / 128) + 8 of them, then 5 + 4 sums: (ceil(cols / 128) + 24) u.
4-bit product: products exact; the tensor core adds the 16 products of one
instruction and the running sum, each addition off by at most 2 u of the larger
magnitude (it may truncate): over the S columns of a scale (16 + S / 16) 2 u.  The
scale's product and its sum round once per S columns, K / S + 1 u in all; parts of K
and of an f32 x (three bf16 values, whose magnitudes sum to at most 1.01 |x|) add 32
sums at most.  Rounding to the result's type adds half a step of it.
"""
import numpy as np

from tests.f8_ref import HALF_STEP, TINY, rounded  # noqa: F401

U = 2.0 ** -24


def route(logits, k, renorm):
    """(idx, weights, tolerance of the weights) by the library's rule: NaN ranks
    above +inf, equal logits by index; a top logit that is not finite gives
    experts 0..k-1 with NaN weights."""
    x = np.asarray(logits, np.float64)
    t, e = x.shape
    rank = np.where(np.isnan(x), np.inf, x)
    idx = np.empty((t, k), np.int64)
    w = np.empty((t, k))
    tol = np.empty((t, k))
    for i in range(t):
        order = sorted(range(e), key=lambda j: (not np.isnan(x[i, j]), -rank[i, j], j))
        idx[i] = order[:k]
        top = x[i, order[0]]
        if not np.isfinite(top):
            idx[i], w[i], tol[i] = np.arange(k), np.nan, 0
            continue
        ex = np.exp(x[i] - top)
        z = ex[idx[i]].sum() if renorm else ex.sum()
        w[i] = ex[idx[i]] / z
        tol[i] = weight_error(x[i], top) * w[i] + 2.0 ** -146
    return idx, w, tol


def weight_error(row, top):
    d = top - row[np.isfinite(row)]
    return (2 * (2 + min(d.max(initial=0), 104.0)) + 38) * U


def route_backward(logits, idx, w, dw, renorm):
    """(gradient, tolerance before rounding)."""
    x, w, dw = (np.asarray(a, np.float64) for a in (logits, w, dw))
    t, e = x.shape
    grad, tol = np.zeros((t, e)), np.zeros((t, e))
    for i in range(t):
        live = [s for s in range(idx.shape[1]) if 0 <= idx[i, s] < e]
        c = sum(w[i, s] * dw[i, s] for s in live)
        C = sum(abs(w[i, s] * dw[i, s]) for s in live)
        if renorm:
            for s in live:
                grad[i, idx[i, s]] += w[i, s] * (dw[i, s] - c)
                tol[i, idx[i, s]] += U * abs(w[i, s]) * (8 * C + 4 * (abs(dw[i, s]) + abs(c)))
            continue
        g, ga = np.zeros(e), np.zeros(e)
        for s in live:
            g[idx[i, s]] += dw[i, s]
            ga[idx[i, s]] += abs(dw[i, s])
        top = np.nan if np.isnan(x[i]).any() else x[i].max()
        if not np.isfinite(top):
            grad[i], tol[i] = np.nan, 0
            continue
        p = np.exp(x[i] - top)
        p /= p.sum()
        grad[i] = p * (g - c)
        tol[i] = (weight_error(x[i], top) + 2 * U) * np.abs(grad[i]) + 2.0 ** -146 * np.abs(g - c) \
            + U * p * (8 * C + 4 * (np.abs(g) + abs(c)) + 16 * ga)
    return grad, tol


def permute(idx, e):
    """(offsets, pos): a stable sort of the pairs by expert."""
    flat = np.asarray(idx).reshape(-1)
    pos = np.full(flat.shape, -1)
    offsets = [0]
    for x in range(e):
        here = np.nonzero(flat == x)[0]
        pos[here] = offsets[-1] + np.arange(len(here))
        offsets.append(offsets[-1] + len(here))
    return np.array(offsets), pos.reshape(np.shape(idx))


def combine(y, pos, w, residual):
    """(out, tolerance before rounding)."""
    t, k = pos.shape
    out = np.zeros((t, y.shape[1])) if residual is None else np.array(residual, np.float64)
    size = np.abs(out)
    for s in range(k):
        r = pos[:, s]
        live = (r >= 0) & (r < y.shape[0])
        term = (1.0 if w is None else w[live, s][:, None]) * y[r[live]]
        out[live] += term
        size[live] += np.abs(term)
    return out, (k + 1) * U * size


def combine_backward(y, pos, w, grad_out, n_rows):
    """(grad_y with NaN where nothing is written, grad_w, tolerance of grad_w)."""
    t, k = pos.shape
    cols = grad_out.shape[1]
    grad_y = np.full((n_rows, cols), np.nan)
    grad_w, tol = np.zeros((t, k)), np.zeros((t, k))
    for s in range(k):
        r = pos[:, s]
        live = (r >= 0) & (r < n_rows)
        grad_y[r[live]] = (1.0 if w is None else w[live, s][:, None]) * grad_out[live]
        prod = y[r[live]] * grad_out[live]
        grad_w[live, s] = prod.sum(1)
        tol[live, s] = (-(-cols // 128) + 24) * U * np.abs(prod).sum(1)
    return grad_y, grad_w, tol


def w4_values(q, scale, zero, group):
    """[..][N][K] values of codes [..][N][K / 2]."""
    codes = np.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1).astype(np.float64)
    z = 8.0 if zero is None else np.repeat((zero & 15).astype(np.float64), group, -1)
    return (codes - z) * np.repeat(np.asarray(scale, np.float64), group, -1)


def w4_product(x, w, group):
    """(y, tolerance before rounding) of x w^T."""
    k = w.shape[1]
    terms = 1.01 * 2 * (16 + group / 16) + k / group + 1 + 32
    return x @ w.T, terms * U * (np.abs(x) @ np.abs(w).T)
