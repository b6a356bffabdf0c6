"""Error bounds of the operators between tokens and singles, from the arithmetic.

As in single_bounds: u = 2^-24 is half a step of fp32, e half a step of the
storage type, a sum of n products in fp32 is off by at most n u times the sum
of their magnitudes, in any order, and exp of x off by d is off by the factor
1 + d. 8 u cover the few operations at each element; the hardware's powers and
logarithms of two are off by one step of fp32 at most.
"""
import numpy as np

import oracle

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
E4M3_HALF = 2.0 ** -4      # of a normal code, relative
E4M3_LEAST_HALF = 2.0 ** -10  # of a subnormal one, in units of the scale


def embedding_bound(out, dtype):
    return (HALF[dtype] + 2 * U) * np.abs(out)


def embedding_backward_bound(tokens, g, vocabulary, scale, old):
    """A sum of a token's rows, the product with the scale, the old value."""
    mag = oracle.embedding_backward(tokens, np.abs(g), vocabulary, abs(scale))
    n = np.bincount([v for v in tokens if 0 <= v < vocabulary], minlength=vocabulary)
    return (n[:, None] + 4) * U * mag + (2 * U * np.abs(old) if old is not None else 0.0)


def norm_bound(y, dtype):
    """A mean of C squares (half of its relative error is the root's), four more
    roundings, the storage's."""
    return (HALF[dtype] + (y.shape[1] / 2 + 8) * U) * np.abs(y)


def norm_backward_bound(h, g_y, w, g_h, g, dtype, eps=1e-6):
    """(bound of g, bound of g_w): sums of C squares and of C products; g_w is a
    sum over rows in fp32 (in stretches) and fp64."""
    T, C = h.shape
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    xhat, gw = np.abs(h * r), np.abs(g_y if w is None else g_y * w)
    mag = r * (gw + xhat * np.mean(gw * xhat, axis=1, keepdims=True))
    more = 0.0 if g_h is None else 2 * U * np.abs(g_h)
    b = HALF[dtype] * np.abs(g) + (2 * C + 24) * U * mag + more
    return b, None if w is None else (C + 16 + T) * U * (np.abs(g_y) * xhat).sum(0)


def _logit_error(x, W, scale, lse):
    """Of logits [rows, V], their magnitudes being up to lse's too."""
    C = x.shape[1]
    mag = abs(scale) * (np.abs(x) @ np.abs(W).T)
    # the exponents are formed in units of log 2: roundings of the logit, of the
    # statistic, of their factors
    return (C + 8) * U * mag + 8 * U * (1.0 + np.abs(lse)[:, None])


def loss_bound(x, W, targets, lse, scale):
    """(bound of nll, bound of lse) of the tokens with a target."""
    live = np.flatnonzero(np.asarray(targets) >= 0)
    bn, bl = np.zeros(len(targets)), np.zeros(len(targets))
    z = scale * (x[live] @ W.T)
    err = _logit_error(x[live], W, scale, lse[live])
    p = np.exp(z - lse[live, None])
    bl[live] = (p * err).sum(1) + (len(W) + 8) * U + 8 * U * (1.0 + np.abs(lse[live]))
    for i, t in enumerate(live):
        if targets[t] < len(W):
            bn[t] = bl[t] + err[i, targets[t]]
    return bn, bl


def loss_backward_bound(x, W, targets, lse, g_nll, g_lse, scale, old, g_x, dtype):
    """(bound of g_x, bound of g_W). d is rounded to the storage type for g_x and kept as
    a pair of bf16, or in fp32, for g_W; either product sums in fp32."""
    live, d, p = oracle.logit_grad(x, W, targets, lse, g_nll, g_lse, scale)
    both = np.abs(g_nll[live]) + (0.0 if g_lse is None else np.abs(g_lse[live]))
    de = both[:, None] * p * (_logit_error(x[live], W, scale, lse[live]) + 8 * U)
    de = de + 4 * U * np.abs(d)
    for i, t in enumerate(live):  # the difference at the target
        de[i, targets[t]] += 4 * U * (both[i] * p[i, targets[t]] + np.abs(g_nll[t]))
    mag, e = np.abs(d), HALF[dtype]
    pair = 2.0 ** -16 if dtype == "bf16" else 0.0
    bx = np.zeros(x.shape)
    s = abs(scale)
    bx[live] = s * ((de + (e + (len(W) + 40) * U) * mag) @ np.abs(W))
    bx = bx + e * np.abs(g_x) + 1e-30
    bW = s * ((de + (pair + (2 * len(live) + 40) * U) * mag).T @ np.abs(x[live])) + 1e-30
    return bx, bW if old is None else bW + 2 * U * np.abs(old)
