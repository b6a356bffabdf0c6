"""GPU tests of attention whose rows' scores all lie near a large number: masks of
-1e9 or of the type's lowest value in every cell, a common offset, large products.
An fp32 log sum does not hold such a row's sum, so gradients that begin with it
weigh every key too much or too little.

The reference is the softmax in 64 bits of scores with the common part taken out
(`small`), which the definition allows. The cases are made so that fp32 holds
every score exactly, or rounds all of a row's to one value; so the only errors are
those of the exponents' differences, of the sums and of the roundings."""
import math

import numpy as np
import pytest

import single_bounds as sb
from gpu_util import announce, bits, f64
from oracle.single import _walk
from test_gpu_single import DT, _dev, _part, _within, nt  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = sb.U
SCALE = 0.125


def _softmax(s):
    top = np.max(s, axis=1, keepdims=True, initial=-np.inf)
    p = np.exp(s - np.where(np.isneginf(top), 0.0, top))
    total = p.sum(1, keepdims=True)
    return p / np.where(total == 0, 1.0, total)


def _reference(rows, cols, small, q, k, v, g, scale, dtype):
    """(values, bounds) of o and the four gradients; small: scores [n, m] by
    (sample's first row, head). The exponent is a difference of scores, exact, in
    units of log 2: off by 4 u of its size, and of the score's where the row keeps
    its log sum; m of them in a sum. P and dS are rounded to the storage type,
    outputs once."""
    H, D = q.shape[1:]
    e = sb.HALF[dtype]
    val = [np.zeros(x.shape) for x in (q, q, k, v)]
    low = [np.zeros(x.shape) for x in (q, q, k, v)]
    cells = sum(n * m for n, m in zip(rows, cols))
    vb, bb = np.zeros((H, cells)), np.zeros((H, cells))
    G_ = H // k.shape[1]
    for r, c, x, n, m, h, kh in _walk(rows, cols, H, k.shape[1]):
        if not n or not m:
            continue
        s = small[r.start, h]
        p = _softmax(s)
        seen = np.where(np.isneginf(s), 0.0, s)
        most = np.abs(seen).max()
        top = np.max(s, axis=1, keepdims=True)
        apart = np.where(np.isneginf(s), 0.0, np.where(np.isneginf(top), 0.0, top) - seen)
        err = 4 * U * (apart + most) + (m + 16) * U
        err = err + (p * err).sum(1, keepdims=True)  # of the power, and of the row's sum
        Q, K, V, G = q[r, h], k[c, kh], v[c, kh], g[r, h]
        O = p @ V  # noqa: E741
        val[0][r, h] = O
        low[0][r, h] = (p * (err + e)) @ np.abs(V) + e * np.abs(O)
        # delta is formed from the stored o
        diff = G @ V.T - (G * O).sum(1, keepdims=True)
        mag = np.abs(G) @ np.abs(V).T + (np.abs(G) * np.abs(O)).sum(1, keepdims=True)
        off = (np.abs(G) * low[0][r, h]).sum(1, keepdims=True)
        ds = p * diff
        de = np.abs(ds) * err + p * ((D + 8) * U * mag + off)
        val[1][r, h] = scale * ds @ K
        low[1][r, h] = abs(scale) * (de + np.abs(ds) * (e + (m + 8) * U)) @ np.abs(K)
        val[2][c, kh] += scale * ds.T @ Q
        low[2][c, kh] += abs(scale) * (de + np.abs(ds) * (e + (G_ * n + 8) * U)).T @ np.abs(Q)
        val[3][c, kh] += p.T @ G
        low[3][c, kh] += (p * (err + e + (G_ * n + 8) * U)).T @ np.abs(G)
        vb[h, x], bb[h, x] = ds.reshape(-1), (de + e * np.abs(ds)).reshape(-1)
    for i in range(1, 4):
        low[i] += e * np.abs(val[i])
    return val + [vb], [b + 1e-30 for b in low + [bb]]


# rows, cols, heads, kv_heads, dim: both walks in one launch; shared key heads, walked one after
# another, by one wave or by several over the same keys; tiles of 128 rows; fp32's own kernels
SHAPES = [
    ([70, 0, 40], None, 2, 2, 32),
    ([70, 33], None, 4, 2, 64),
    ([130, 5], None, 2, 2, 96),
    ([3, 1, 65], [90, 64, 130], 4, 1, 40),
    ([200], None, 2, 1, 128),
    ([32] * 256 + [70], None, 8, 8, 16),
]


def _large_products(rng, rows, cols, H, K, D, dtype, sign):
    """q, k (device, 64 bits) and, by sample and head, the scores without their common
    part, causal, with that part of every row: one dimension adds 2^17 to the odd
    rows' scores (or takes it away), the others steps of 1/8. Products and sums
    are exact in fp32, and so is their maximum times the scale."""
    c = cols or rows
    T, Tc = sum(rows), sum(c)
    a, b = (rng.integers(-1, 2, size=s).astype(float) for s in ((T, H, D), (Tc, K, D)))
    a[:, :, 0], b[:, :, 0] = 0.0, 2.0 ** 10
    a[1::2, :, 0] = sign * 2.0 ** 10
    (q, q64), (k, k64) = _dev(a, dtype), _dev(b, dtype)
    small = {}
    for r, cc, x, n, m, h, kh in _walk(rows, c, H, K):
        if n and m:
            s = SCALE * q64[r, h, 1:] @ k64[cc, kh, 1:].T
            small[r.start, h] = np.where(np.arange(m)[None] > np.arange(n)[:, None] + m - n,
                                         -np.inf, s)
    return q, q64, k, k64, small, SCALE * q64[:, :, 0] * 2.0 ** 10


SPLIT = [([1, 1, 0, 2, 1], [5000, 1, 700, 64, 3001], 8, 2, 64), ([150, 3], [2100, 40], 2, 1, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("shape", SHAPES + SPLIT)
def test_large_products(nt, shape, sign, dtype):  # noqa: F811
    """Without a bias. Bases that move, waves and parts that are joined, each with a
    maximum of its own, weigh their keys alike. The log sum is rounded once where the
    maximum and the sum's logarithm are added."""
    rows, cols, H, K, D = shape
    announce(f"attention large products {shape} {sign} {dtype}"[:200])
    rng = np.random.default_rng(62)
    c = cols or rows
    q, q64, k, k64, small, common = _large_products(rng, rows, cols, H, K, D, dtype, sign)
    (v, v64), (g, g64) = (_dev(rng.normal(size=s), dtype) for s in ((sum(c), K, D), (sum(rows), H, D)))
    p = _part(nt, rows, cols)
    o, lse = nt.nt_single_attention(p, q, k, v, causal=True, scale=SCALE)
    torch.cuda.synchronize()
    val, low = _reference(rows, c, small, q64, k64, v64, g64, SCALE, dtype)
    _within("o", f64(o, torch), val[0], low[0])
    z, e = np.full(common.shape, -np.inf), np.zeros(common.shape)
    for (start, h), s in small.items():
        top = s.max(1)
        at = np.where(np.isneginf(top), 0.0, top)
        with np.errstate(divide="ignore"):
            z[start:start + len(s), h] = at + np.log(np.exp(s - at[:, None]).sum(1))
        e[start:start + len(s), h] = (s.shape[1] + 32 + 8 * np.abs(at)) * U
    z = z + common
    _within("lse", f64(lse, torch), z, e + 4 * U * np.abs(np.where(np.isfinite(z), z, 0.0)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_masks_and_offsets_of_whole_rows(nt, shape, causal, dtype):  # noqa: F811
    """Every fifth row: all cells at the lowest value; at -2^30 (a score below 32
    vanishes beside it); at an offset of -2^20, or of 2^20, beside which fp32 holds
    steps of 1/8; nothing at all; then an ordinary row."""
    rows, cols, H, K, D = shape
    announce(f"attention offsets {shape} {causal} {dtype}"[:200])
    rng = np.random.default_rng(61)
    c = cols or rows
    T, Tc, cells = sum(rows), sum(c), sum(n * m for n, m in zip(rows, c))
    lowest = float(torch.finfo(getattr(torch, DT[dtype])).min)
    kinds = [lowest, -2.0 ** 30, -2.0 ** 20, 2.0 ** 20, -math.inf, 0.0]
    (q, q64), (k, k64) = (_dev(rng.integers(-1, 2, size=s), dtype) for s in ((T, H, D), (Tc, K, D)))
    (v, v64), (g, g64) = (_dev(rng.normal(size=s), dtype) for s in ((Tc, K, D), (T, H, D)))
    b = np.zeros((H, cells))
    small = {}
    for r, cc, x, n, m, h, kh in _walk(rows, c, H, K):
        if not n or not m:
            continue
        s = SCALE * q64[r, h] @ k64[cc, kh].T
        at = np.array([kinds[(i + h) % 6] for i in range(n)])
        b[h, x] = np.repeat(at, m)
        s = np.where((np.abs(at) > 2.0 ** 25)[:, None], 0.0, s)  # all of them one value
        s = np.where(np.isneginf(at)[:, None], -np.inf, s)
        if causal:
            s = np.where(np.arange(m)[None] > np.arange(n)[:, None] + m - n, -np.inf, s)
        small[r.start, h] = s
    bias, _ = _dev(b, dtype)
    p = _part(nt, rows, cols)
    o, lse = nt.nt_single_attention(p, q, k, v, bias=bias, causal=causal, scale=SCALE)
    need = nt.nt_attention_backward_workspace_bytes(p, H, K, D, q.dtype, causal)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    call = lambda: nt.nt_single_attention_backward(  # noqa: E731
        p, q, k, v, o, lse, g, bias=bias, causal=causal, scale=SCALE, workspace=ws)
    got, again = call(), call()
    torch.cuda.synchronize()
    val, low = _reference(rows, c, small, q64, k64, v64, g64, SCALE, dtype)
    for name, x, r, e in zip(("o", "g_q", "g_k", "g_v", "g_bias"), (o,) + got, val, low):
        _within(name, f64(x, torch), r, e)
    for x, y in zip(got, again):
        np.testing.assert_array_equal(bits(x, torch), bits(y, torch))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("shape", SHAPES)
def test_large_products_gradient(nt, shape, sign, dtype):  # noqa: F811
    rows, cols, H, K, D = shape
    announce(f"attention gradient, large products {shape} {sign} {dtype}"[:200])
    rng = np.random.default_rng(63)
    c = cols or rows
    q, q64, k, k64, small, _ = _large_products(rng, rows, cols, H, K, D, dtype, sign)
    (v, v64), (g, g64) = (_dev(rng.normal(size=s), dtype) for s in ((sum(c), K, D), (sum(rows), H, D)))
    p = _part(nt, rows, cols)
    o, lse = nt.nt_single_attention(p, q, k, v, causal=True, scale=SCALE)
    got = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, causal=True, scale=SCALE)
    torch.cuda.synchronize()
    val, low = _reference(rows, c, small, q64, k64, v64, g64, SCALE, dtype)
    for name, x, r, e in zip(("o", "g_q", "g_k", "g_v"), (o,) + got, val, low):
        _within(name, f64(x, torch), r, e)
