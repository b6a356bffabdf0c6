"""Single attention, norms with rotation, and AdamW: float64 from the
definitions, sample by sample and head by head, with no rounding.
"""
import math

import numpy as np


# ------------------------------------------------------------------ rotation
def rotary_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original=0.0,
                       beta_fast=32.0, beta_slow=1.0):
    """Angle per position of each of the rot_dim / 2 pairs."""
    out = []
    for j in range(rot_dim // 2):
        f = base ** (-2.0 * j / rot_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "parts":
            turns = original * f / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)))
            f = f * keep + f / factor * (1.0 - keep)
        out.append(f)
    return np.array(out)


def rotary_table(positions, rot_dim, magnitude=1.0, **scaling):
    a = np.arange(positions)[:, None] * rotary_frequencies(rot_dim, **scaling)[None]
    return np.concatenate([np.cos(a), np.sin(a)], 1) * magnitude


def rotation_matrix(row, head_dim, interleaved):
    """The head_dim x head_dim matrix of one position's table row."""
    R = len(row)
    m = np.eye(head_dim)
    for j in range(R // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)
        c, s = row[j], row[R // 2 + j]
        m[a, a], m[a, b], m[b, a], m[b, b] = c, -s, s, c
    return m


def positions_of(lengths):
    return np.concatenate([np.arange(n) for n in lengths] + [np.zeros(0)]).astype(np.int64)


def norm_rotary(x, w, table, positions, interleaved=False, eps=1e-6):
    """x [T, h, D]; w [D] or None; table or None. Norm, then rotation."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * w
    if table is None:
        return y
    for t, at in enumerate(positions):
        y[t] = y[t] @ rotation_matrix(table[at], y.shape[-1], interleaved).T
    return y


def norm_rotary_backward(x, g, w, table, positions, interleaved=False, eps=1e-6):
    """(g_x, g_w) for the output's gradient g; g_w None without w."""
    h = np.array(g, dtype=np.float64)
    if table is not None:
        for t, at in enumerate(positions):
            h[t] = h[t] @ rotation_matrix(table[at], h.shape[-1], interleaved)
    if w is None:
        return h, None
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    xhat = x * r
    hw = h * w
    return r * (hw - xhat * np.mean(hw * xhat, axis=-1, keepdims=True)), \
        np.sum(h * xhat, axis=(0, 1))


# ----------------------------------------------------------------- attention
def _scores(q, k, bias, scale, causal):
    n, m = len(q), len(k)
    s = scale * (q @ k.T)
    if bias is not None:
        s = s + bias
    if causal:
        hidden = np.arange(m)[None] > np.arange(n)[:, None] + m - n
        s = np.where(hidden, -np.inf, s)
    return s


def _walk(rows, cols, heads, kv_heads):
    """(row slice, column slice, cell slice, n, m, head, key head)."""
    a = b = cell = 0
    for n, m in zip(rows, cols):
        for h in range(heads):
            yield (slice(a, a + n), slice(b, b + m), slice(cell, cell + n * m), n, m, h,
                   h // (heads // kv_heads))
        a, b, cell = a + n, b + m, cell + n * m


def attention(rows, cols, q, k, v, bias=None, causal=False, scale=1.0):
    """(o, lse): q [T, H, D], k, v [T_cols, K, D], bias [H, cells]."""
    H = q.shape[1]
    o, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    for r, c, x, n, m, h, kh in _walk(rows, cols, H, k.shape[1]):
        s = _scores(q[r, h], k[c, kh], None if bias is None else bias[h, x].reshape(n, m), scale,
                    causal)
        for i in range(n):
            if m == 0 or np.all(np.isneginf(s[i])):
                continue
            top = np.max(s[i])
            p = np.exp(s[i] - top)
            o[r.start + i, h] = p @ v[c, kh] / np.sum(p)
            lse[r.start + i, h] = top + math.log(np.sum(p))
    return o, lse


def attention_backward(rows, cols, q, k, v, o, lse, g_o, bias=None, causal=False, scale=1.0):
    """(g_q, g_k, g_v, g_bias) from the given o and lse."""
    H = q.shape[1]
    g_q, g_k, g_v = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    g_bias = None if bias is None else np.zeros(bias.shape)
    for r, c, x, n, m, h, kh in _walk(rows, cols, H, k.shape[1]):
        if n == 0 or m == 0:
            continue
        p = _probabilities(q[r, h], k[c, kh], bias, lse[r, h], h, x, n, m, scale, causal)
        delta = np.sum(g_o[r, h] * o[r, h], axis=1, keepdims=True)
        ds = p * (g_o[r, h] @ v[c, kh].T - delta)
        g_v[c, kh] += p.T @ g_o[r, h]
        g_q[r, h] = scale * ds @ k[c, kh]
        g_k[c, kh] += scale * ds.T @ q[r, h]
        if bias is not None:
            g_bias[h, x] = ds.reshape(-1)
    return g_q, g_k, g_v, g_bias


def _probabilities(q, k, bias, lse, h, x, n, m, scale, causal):
    s = _scores(q, k, None if bias is None else bias[h, x].reshape(n, m), scale, causal)
    z = lse[:, None]
    return np.where(np.isneginf(z) | np.isneginf(s), 0.0,
                    np.exp(np.where(np.isneginf(s), 0.0, s) - np.where(np.isneginf(z), 0.0, z)))


# -------------------------------------------------------------------- update
def adamw(w, g, m, v, step, lr, beta1, beta2, eps, weight_decay):
    """(w, m, v) after one step."""
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    mhat, vhat = m / (1.0 - beta1 ** step), v / (1.0 - beta2 ** step)
    return w - lr * weight_decay * w - lr * mhat / (np.sqrt(vhat) + eps), m, v


def e4m3_values():
    """The finite values of the 256 codes (NaN for the two codes without one)."""
    out = []
    for code in range(256):
        sign, e, f = -1.0 if code & 128 else 1.0, (code >> 3) & 15, code & 7
        if e == 15 and f == 7:
            out.append(math.nan)
        else:
            out.append(sign * (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)))
    return np.array(out)


def block_scales(x, block=256):
    """The largest magnitude of each block over 448 (finite values only)."""
    x = np.where(np.isfinite(x), x, 0.0)
    return np.array([np.max(np.abs(x[i:i + block])) / 448.0 for i in range(0, len(x), block)])
