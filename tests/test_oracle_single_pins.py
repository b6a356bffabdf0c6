"""Pins of the single attention oracle and the AdamW oracle (no GPU): scalar
loops, closed forms, central differences of the forward functions, and torch's
own e4m3 type."""
import math

import numpy as np
import pytest

import oracle


def test_rotation_turns_pairs():
    table = oracle.rotary_table(5, 4)
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    for inter, (a, b), (c, d) in ((False, (0, 2), (1, 3)), (True, (0, 1), (2, 3))):
        y = oracle.norm_rotary(x, None, table, [3], inter)[0, 0]
        z = [complex(x[0, 0, a], x[0, 0, b]) * np.exp(3j),
             complex(x[0, 0, c], x[0, 0, d]) * np.exp(3j * 10000.0 ** -0.5)]
        np.testing.assert_allclose([y[a], y[b], y[c], y[d]],
                                   [z[0].real, z[0].imag, z[1].real, z[1].imag], rtol=1e-14)
        np.testing.assert_array_equal(y[4:], x[0, 0, 4:])


def test_rotary_scalings():
    plain = oracle.rotary_frequencies(64)
    np.testing.assert_allclose(oracle.rotary_frequencies(64, scaling="linear", factor=4.0), plain / 4)
    f = oracle.rotary_frequencies(64, scaling="parts", factor=4.0, original=2048.0)
    turns = 2048.0 * plain / (2 * math.pi)
    np.testing.assert_allclose(f[turns >= 32], plain[turns >= 32])
    np.testing.assert_allclose(f[turns <= 1], plain[turns <= 1] / 4)
    assert np.all(np.diff(f) < 0)


def test_scores_depend_on_the_distance_only():
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(2, 1, 1, 16))
    table = oracle.rotary_table(40, 16)
    dot = lambda a, b: float(np.sum(oracle.norm_rotary(q, None, table, [a]) *  # noqa: E731
                                    oracle.norm_rotary(k, None, table, [b])))
    assert abs(dot(7, 3) - dot(36, 32)) < 1e-12


def _numeric(f, x, h=1e-6):
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


@pytest.mark.parametrize("inter", [False, True])
def test_norm_backward_by_differences(inter):
    rng = np.random.default_rng(2)
    x, g, w = rng.normal(size=(3, 2, 8)), rng.normal(size=(3, 2, 8)), 1 + 0.1 * rng.normal(size=8)
    table, at = oracle.rotary_table(9, 6), [0, 4, 8]
    loss = lambda y, u: float(np.sum(g * oracle.norm_rotary(y, u, table, at, inter)))  # noqa: E731
    gx, gw = oracle.norm_rotary_backward(x, g, w, table, at, inter)
    np.testing.assert_allclose(gx, _numeric(lambda y: loss(y, w), x), atol=1e-8)
    np.testing.assert_allclose(gw, _numeric(lambda u: loss(x, u), w), atol=1e-8)


@pytest.mark.parametrize("causal", [False, True])
def test_attention_by_scalar_loops(causal):
    rng = np.random.default_rng(3)
    rows, cols, H, K, D = [2, 0, 3, 1], [3, 2, 2, 0], 4, 2, 8
    q, k, v = rng.normal(size=(6, H, D)), rng.normal(size=(7, K, D)), rng.normal(size=(7, K, D))
    bias = rng.normal(size=(H, 12))
    bias[:, 4] = -np.inf
    o, lse = oracle.attention(rows, cols, q, k, v, bias, causal, 0.3)
    a = b = cell = 0
    for n, m in zip(rows, cols):
        for r in range(n):
            for h in range(H):
                w = {}
                for c in range(m):
                    if causal and c > r + m - n:
                        continue
                    w[c] = math.exp(0.3 * sum(q[a + r, h, d] * k[b + c, h // 2, d] for d in range(D))
                                    + bias[h, cell + r * m + c])
                total = sum(w.values())
                want = [sum(x * v[b + c, h // 2, d] for c, x in w.items()) / total if total else 0.0
                        for d in range(D)]
                np.testing.assert_allclose(o[a + r, h], want, atol=1e-13)
                assert lse[a + r, h] == (pytest.approx(math.log(total)) if total else -np.inf)
        a, b, cell = a + n, b + m, cell + n * m


@pytest.mark.parametrize("causal", [False, True])
def test_attention_backward_by_differences(causal):
    rng = np.random.default_rng(4)
    rows, cols, H, K, D = [3, 2], [2, 4], 2, 1, 8
    xs = [rng.normal(size=s) for s in ((5, H, D), (6, K, D), (6, K, D), (H, 14))]
    g = rng.normal(size=(5, H, D))

    def loss(*ys):
        return float(np.sum(g * oracle.attention(rows, cols, *ys, causal, 0.4)[0]))

    o, lse = oracle.attention(rows, cols, *xs, causal, 0.4)
    grads = oracle.attention_backward(rows, cols, *xs[:3], o, lse, g, xs[3], causal, 0.4)
    for i in range(4):
        num = _numeric(lambda y: loss(*[y if j == i else x for j, x in enumerate(xs)]), xs[i])
        np.testing.assert_allclose(grads[i], num, atol=1e-8)


def test_attention_empty_rows():
    rng = np.random.default_rng(5)
    q, k, v = rng.normal(size=(3, 1, 8)), rng.normal(size=(2, 1, 8)), rng.normal(size=(2, 1, 8))
    bias = np.zeros((1, 6))
    bias[0, 2:4] = -np.inf
    o, lse = oracle.attention([3], [2], q, k, v, bias)
    assert np.all(o[1] == 0) and np.isneginf(lse[1, 0])
    grads = oracle.attention_backward([3], [2], q, k, v, o, lse, np.ones((3, 1, 8)), bias)
    assert np.all(grads[0][1] == 0) and all(np.isfinite(x).all() for x in grads)


def test_adamw_first_step_and_decay():
    w, g = np.array([1.0, -2.0]), np.array([0.5, -3.0])
    new, m, v = oracle.adamw(w, g, 0.0, 0.0, 1, 0.1, 0.9, 0.999, 0.0, 0.0)
    np.testing.assert_allclose(new, w - 0.1 * np.sign(g))  # the corrected first step is the sign
    np.testing.assert_allclose(m, 0.1 * g)
    np.testing.assert_allclose(v, 0.001 * g * g)
    new, _, _ = oracle.adamw(w, 0 * g, 0.0, 0.0, 1, 0.1, 0.9, 0.999, 1e-8, 0.5)
    np.testing.assert_allclose(new, w * 0.95)


def test_e4m3_values_are_torchs():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(oracle.e4m3_values(), t.astype(np.float64))
    x = np.arange(600.0)
    x[599] = np.inf
    np.testing.assert_allclose(oracle.block_scales(x), np.array([255, 511, 598]) / 448)
