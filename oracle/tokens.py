"""Embedding of tokens, the norm with the residual, and the cross entropy over a
vocabulary: float64 from the definitions, token by token or in whole matrices,
with no rounding.
"""
import numpy as np


def embedding(table, tokens, scale=1.0):
    """Absent tokens (< 0) give zeros, tokens that the table does not hold NaN."""
    out = np.zeros((len(tokens), table.shape[1]))
    for t, v in enumerate(tokens):
        if v >= len(table):
            out[t] = np.nan
        elif v >= 0:
            out[t] = scale * table[v]
    return out


def embedding_backward(tokens, g, vocabulary, scale=1.0, old=None):
    out = np.zeros((vocabulary, g.shape[1])) if old is None else np.array(old, dtype=np.float64)
    for t, v in enumerate(tokens):
        if 0 <= v < vocabulary:
            out[v] += scale * g[t]
    return out


def residual_norm(h, w=None, eps=1e-6):
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return y if w is None else y * w


def residual_norm_backward(h, g_y, w=None, g_h=None, eps=1e-6):
    """(g, g_w): the adjoint of y_c = h_c w_c r(h), r = (mean h^2 + eps)^(-1/2),
    from dr/dh_c = -r^3 h_c / C."""
    r = (np.mean(h * h, axis=1, keepdims=True) + eps) ** -0.5
    gw = g_y if w is None else g_y * w
    g = gw * r - (gw * h).sum(1, keepdims=True) * r ** 3 * h / h.shape[1]
    if g_h is not None:
        g = g + g_h
    return g, None if w is None else (g_y * h * r).sum(0)


def token_loss(x, W, targets, scale=1.0):
    """(nll, lse); tokens whose target is below zero are zeros in both, and a
    target that the vocabulary does not hold has nll NaN."""
    nll, lse = np.zeros(len(targets)), np.zeros(len(targets))
    for t, v in enumerate(targets):
        if v >= 0:
            z = scale * (W @ x[t])
            top = z.max()
            lse[t] = top if np.isinf(top) else top + np.log(np.exp(z - top).sum())
            nll[t] = lse[t] - z[v] if v < len(W) else np.nan
    return nll, lse


def logit_grad(x, W, targets, lse, g_nll, g_lse=None, scale=1.0):
    """(rows with a target, d of them [rows, vocabulary], their probabilities)."""
    live = np.flatnonzero(np.asarray(targets) >= 0)
    p = np.exp(scale * (x[live] @ W.T) - lse[live, None])
    both = g_nll[live] if g_lse is None else g_nll[live] + g_lse[live]
    d = p * both[:, None]
    for i, t in enumerate(live):
        if targets[t] < len(W):
            d[i, targets[t]] -= g_nll[t]
        else:
            d[i] = np.nan
    return live, d, p


def token_loss_backward(x, W, targets, lse, g_nll, g_lse=None, scale=1.0, old=None):
    """(g_x, g_W)."""
    live, d, _ = logit_grad(x, W, targets, lse, g_nll, g_lse, scale)
    g_x = np.zeros(x.shape)
    g_x[live] = scale * (d @ W)
    g_W = scale * (d.T @ x[live])
    return g_x, g_W if old is None else old + g_W
