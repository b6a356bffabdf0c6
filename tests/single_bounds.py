"""Error bounds of the single attention operators, from the arithmetic.

u = 2^-24 is half a step of fp32, e half a step of the storage type (bf16
2^-8, fp32 2^-24). A sum of n products in fp32 is off by at most n u times
the sum of their magnitudes, in any order; exp of x off by d is off by the
factor 1 + d. Each bound adds up the roundings on the way of one value, with
8 u for the few operations at each element.
"""
import numpy as np

from oracle.single import _probabilities, _scores, _walk

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def norm_bound(x, w, out, table, dtype):
    """The norm: a mean of D squares and ten more operations on each value;
    the rotation: two products and a sum of its pair. The pair's magnitudes
    are at most the row's largest."""
    D = x.shape[-1]
    y = np.abs(out).max(axis=-1, keepdims=True)
    if table is not None:
        y = y + np.abs(out).max(axis=-1, keepdims=True) * 0.5
    return HALF[dtype] * np.abs(out) + (D + 16) * U * 2.0 * y


def norm_backward_bound(x, w, g, g_x, dtype):
    """(bound of g_x, bound of g_w): h = the gradient turned back (a pair's
    magnitude is kept), times w; a mean of D products; g_w sums tokens x heads
    terms, in fp32 over at most 2^12 of them and in fp64 beyond."""
    D = x.shape[-1]
    h = np.abs(g).max(axis=-1, keepdims=True) * 1.5
    if w is None:
        return HALF[dtype] * np.abs(g_x) + 4 * U * h, None
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + 1e-6)
    xhat = np.abs(x * r)
    hw = h * np.abs(w).max()
    mag = r * (hw + xhat * np.mean(hw * xhat, axis=-1, keepdims=True))
    terms = min(x.shape[0] * x.shape[1], 4096)
    return HALF[dtype] * np.abs(g_x) + (2 * D + 24) * U * mag, \
        (D + 16 + terms) * U * (h * xhat).sum((0, 1))


def _score_error(q, k, bias, scale, D):
    """Of a score, and of exp of its difference to a row's statistic."""
    mag = scale * (np.abs(q) @ np.abs(k).T)
    if bias is not None:
        mag = mag + np.where(np.isfinite(bias), np.abs(bias), 0.0)
    # the exponent is formed in units of log 2: one more rounding of the score and of
    # the statistic, which is at most the largest magnitude
    return (D + 8) * U * mag + 8 * U * (1.0 + mag.max(axis=1, keepdims=True, initial=0.0))


def attention_bound(rows, cols, q, k, v, o, lse, bias, causal, scale, dtype):
    """(bound of o, bound of lse)."""
    H, D = q.shape[1:]
    bo, bl = np.zeros(o.shape), np.zeros(lse.shape)
    for r, c, x, n, m, h, kh in _walk(rows, cols, H, k.shape[1]):
        if not n or not m:
            continue
        b = None if bias is None else bias[h, x].reshape(n, m)
        p = _probabilities(q[r, h], k[c, kh], bias, lse[r, h], h, x, n, m, scale, causal)
        err = _score_error(q[r, h], k[c, kh], b, scale, D) + (m + 8) * U
        mean = (p * err).sum(1, keepdims=True)  # of the sum of the probabilities
        # probabilities are rounded to the storage type before their product
        bo[r, h] = (p * (err + mean + HALF[dtype])) @ np.abs(v[c, kh]) + HALF[dtype] * np.abs(o[r, h])
        bl[r, h] = mean[:, 0] + 8 * U * (1.0 + np.abs(np.where(np.isfinite(lse[r, h]), lse[r, h], 0)))
    return bo + 1e-30, bl


def attention_backward_bound(rows, cols, q, k, v, o, lse, g_o, grads, bias, causal, scale, dtype):
    """Bounds of (g_q, g_k, g_v, g_bias)."""
    H, D = q.shape[1:]
    e = HALF[dtype]
    bq, bk, bv = (np.zeros(t.shape) for t in (q, k, v))
    bb = None if bias is None else np.zeros(bias.shape)
    for r, c, x, n, m, h, kh in _walk(rows, cols, H, k.shape[1]):
        if not n or not m:
            continue
        b = None if bias is None else bias[h, x].reshape(n, m)
        Q, K, V, O, G = q[r, h], k[c, kh], v[c, kh], o[r, h], g_o[r, h]
        p = _probabilities(Q, K, bias, lse[r, h], h, x, n, m, scale, causal)
        z = np.where(np.isfinite(lse[r, h]), np.abs(lse[r, h]), 0.0)[:, None]
        dp = _score_error(Q, K, b, scale, D) + 8 * U * (1.0 + z)
        diff = G @ V.T - (G * O).sum(1, keepdims=True)
        mag = np.abs(G) @ np.abs(V).T + (np.abs(G) * np.abs(O)).sum(1, keepdims=True)
        ds = np.abs(p * diff)
        de = ds * dp + p * (D + 8) * U * mag  # of dS before its rounding
        G_ = H // k.shape[1]
        bv[c, kh] += (p * (dp + e + (G_ * n + 8) * U)).T @ np.abs(G)
        # scale joins dS or the product: one rounding either way
        bq[r, h] = scale * (de + ds * (e + (m + 8) * U)) @ np.abs(K)
        bk[c, kh] += scale * (de + ds * (e + (G_ * n + 8) * U)).T @ np.abs(Q)
        if bias is not None:
            bb[h, x] = (de + e * ds).reshape(-1)
    bq, bk, bv = (b + e * np.abs(g) + 1e-30 for b, g in zip((bq, bk, bv), grads))
    return bq, bk, bv, None if bb is None else bb + 1e-30


__all__ = ["U", "HALF", "norm_bound", "attention_bound", "attention_backward_bound", "_scores"]
