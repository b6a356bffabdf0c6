"""Pins of the oracle of the operators between tokens and singles (no GPU):
closed forms and central differences of the forward functions."""
import numpy as np

import oracle


def test_embedding_rows():
    table = np.arange(12.0).reshape(3, 4)
    out = oracle.embedding(table, [2, -1, 0, 3], 0.5)
    np.testing.assert_array_equal(out[:3], [[4, 4.5, 5, 5.5], [0] * 4, [0, 0.5, 1, 1.5]])
    assert np.isnan(out[3]).all()


def test_embedding_backward_is_the_adjoint():
    """<g, E(table)> = <E^T(g), table>, and what is there stays added."""
    rng = np.random.default_rng(0)
    table, g, old = rng.normal(size=(7, 8)), rng.normal(size=(20, 8)), rng.normal(size=(7, 8))
    ids = rng.integers(-1, 7, size=20)
    back = oracle.embedding_backward(ids, g, 7, 1.5)
    np.testing.assert_allclose((g * oracle.embedding(table, ids, 1.5)).sum(), (back * table).sum())
    np.testing.assert_allclose(oracle.embedding_backward(ids, g, 7, 1.5, old), old + back)
    assert (oracle.embedding_backward([7, -3], g[:2], 7) == 0).all()


def test_norm_of_a_constant_row():
    y = oracle.residual_norm(np.full((1, 8), -3.0), np.arange(8.0), eps=0.0)
    np.testing.assert_allclose(y[0], -np.arange(8.0))


def _differences(f, x, step=1e-6):
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + step
        up = f()
        x[i] = keep - step
        g[i] = (up - f()) / (2 * step)
        x[i] = keep
    return g


def test_norm_backward_against_differences():
    rng = np.random.default_rng(1)
    h, g_y, g_h = rng.normal(size=(3, 4, 8))
    w = rng.normal(size=8)

    def value():
        return (oracle.residual_norm(h, w, 1e-2) * g_y).sum() + (h * g_h).sum()

    g, g_w = oracle.residual_norm_backward(h, g_y, w, g_h, 1e-2)
    np.testing.assert_allclose(g, _differences(value, h), atol=1e-8)
    np.testing.assert_allclose(g_w, _differences(value, w), atol=1e-8)
    np.testing.assert_allclose(oracle.residual_norm_backward(h, g_y, None, None, 1e-2)[0],
                               oracle.residual_norm_backward(h, g_y, np.ones(8), None, 1e-2)[0])


def test_loss_of_equal_logits():
    nll, lse = oracle.token_loss(np.zeros((3, 4)), np.ones((10, 4)), [3, -1, 10])
    np.testing.assert_allclose(lse, [np.log(10), 0, np.log(10)])
    np.testing.assert_allclose(nll[:2], [np.log(10), 0])
    assert np.isnan(nll[2])


def test_loss_backward_against_differences():
    rng = np.random.default_rng(2)
    x, W = rng.normal(size=(5, 6)), rng.normal(size=(7, 6))
    ids, a, b, scale = np.array([0, 6, -1, 3, 3]), rng.normal(size=5), rng.normal(size=5), 0.7

    def value():
        nll, lse = oracle.token_loss(x, W, ids, scale)
        return nll @ a + lse @ b

    lse = oracle.token_loss(x, W, ids, scale)[1]
    old = rng.normal(size=W.shape)
    g_x, g_W = oracle.token_loss_backward(x, W, ids, lse, a, b, scale, old)
    np.testing.assert_allclose(g_x, _differences(value, x), atol=1e-8)
    np.testing.assert_allclose(g_W - old, _differences(value, W), atol=1e-8)
    assert (g_x[2] == 0).all()
