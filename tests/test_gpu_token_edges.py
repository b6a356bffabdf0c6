"""GPU tests of the operators between tokens and singles where they can go wrong:
precision next to a rounding, the smallest numbers, the pieces and tiles that a
batch's sizes lead to, paths that keep state in a workspace."""
import math

import numpy as np
import pytest

import oracle
import token_bounds as tb
from gpu_util import announce, bits, f64
from token_cases import LOSS_PLANS
from test_gpu_token import _check_loss, _dev, _ids, _loss_inputs, _within, nt  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ----------------------------------------------------------- loss's gradient
def _pair_bound(x, W, ids, lse, g_nll, g_lse, scale, old, g_x, dtype):
    """(bound of g_x, bound of g_W) where both products take d as a pair of bf16: hi
    leaves at most 2^-8 of d and lo 2^-8 of that. As token_bounds.loss_backward_bound
    for the logits and sums (each product twice as many terms); beside them g_x has the
    one rounding of its storage."""
    live, d, p = oracle.logit_grad(x, W, ids, lse, g_nll, g_lse, scale)
    both = np.abs(g_nll[live]) + (0.0 if g_lse is None else np.abs(g_lse[live]))
    de = both[:, None] * p * (tb._logit_error(x[live], W, scale, lse[live]) + 8 * tb.U)
    de = de + 4 * tb.U * np.abs(d)
    for i, t in enumerate(live):
        de[i, ids[t]] += 4 * tb.U * (both[i] * p[i, ids[t]] + np.abs(g_nll[t]))
    pair = 2.0 ** -16 if dtype == "bf16" else 0.0
    bx = np.zeros(x.shape)
    bx[live] = abs(scale) * ((de + (pair + (2 * len(W) + 40) * tb.U) * np.abs(d)) @ np.abs(W))
    bx = (1 + 2.0 ** -8) * bx + tb.HALF[dtype] * np.abs(g_x) + 1e-30
    bW = abs(scale) * ((de + (pair + (2 * len(live) + 40) * tb.U) * np.abs(d)).T
                       @ np.abs(x[live])) + 1e-30
    return bx, bW if old is None else bW + 2 * tb.U * np.abs(old)


def _check_gradients(nt, x, x64, W, W64, ids, lse, dtype, rng, scale=1.0, both=False,
                     accumulate=False):
    T = len(ids)
    g_nll, gn64 = _dev(rng.normal(size=T) / T)
    g_lse, gl64 = _dev(rng.normal(size=T) / T) if both else (None, None)
    old, old64 = _dev(rng.normal(size=W64.shape) * 1e-2) if accumulate else (None, None)
    g_x, g_W = nt.nt_token_loss_backward(x, W, _ids(ids), lse, g_nll, g_lse=g_lse, scale=scale,
                                         g_W=old, accumulate=accumulate)
    s, l64 = np.float64(np.float32(scale)), f64(lse, torch)
    rx, rW = oracle.token_loss_backward(x64, W64, ids, l64, gn64, gl64, s, old64)
    bx, bW = _pair_bound(x64, W64, ids, l64, gn64, gl64, s, old64, rx, dtype)
    _within("g_x", g_x, rx, bx)
    _within("g_W", g_W, rW, bW)
    return g_nll, g_lse, g_x, g_W


@pytest.mark.parametrize("T,V,C", [(1, 300, 64), (33, 33, 8), (40, 2000, 64), (130, 300, 200),
                                   (257, 128, 1032), (300, 1301, 128)])
def test_loss_gradient_beside_one_rounding(nt, T, V, C):
    """In bf16 g_x is off by its own rounding and next to nothing else: where the terms of
    its sum cancel, one rounding of them would be seen."""
    announce(f"loss backward, pair, T={T} V={V} C={C}")
    rng = np.random.default_rng(T + V)
    x, x64, W, W64, ids = _loss_inputs(rng, T, V, C, "bf16")
    for scale, both in ((1.0, False), (-0.3, True)):
        lse = nt.nt_token_loss(x, W, _ids(ids), scale=scale)[1]
        _check_gradients(nt, x, x64, W, W64, ids, lse, "bf16", rng, scale, both, both)


def test_loss_gradient_at_the_target(nt):
    """d at the target dominates: hardly any probability elsewhere, the target's row of W
    large, and d there (p - 1) g with a g that bf16 does not hold."""
    T, V, C = 60, 200, 64
    announce("loss backward, d at the target")
    rng = np.random.default_rng(1)
    x, x64 = _dev(rng.normal(size=(T, C)) * 1e-3, "bf16")
    W, W64 = _dev(rng.normal(size=(V, C)) * 100, "bf16")
    ids = rng.integers(0, V, size=T)
    lse = nt.nt_token_loss(x, W, _ids(ids))[1]
    _check_gradients(nt, x, x64, W, W64, ids, lse, "bf16", rng)


@pytest.mark.parametrize("name", LOSS_PLANS)
def test_loss_of_many(nt, name):
    """Large tiles with partial ones at both ends, pieces of the vocabulary with a short last
    one (parts of whose rows are empty), passes over the tokens: forward and both gradients,
    with targets in every piece, added to an old one."""
    T, V, C, dtype, absent, said = LOSS_PLANS[name]
    announce(f"loss of many, {name}: T={T} V={V} C={C} {dtype}")
    rng = np.random.default_rng(T + V)
    x, x64, W, W64, ids = _loss_inputs(rng, T, V, C, dtype, absent=absent)
    piece, pieces = said.get("piece", 1024), said.get("pieces", 1)
    if pieces > 1:  # the first and the last word of every piece
        edges = np.r_[np.arange(pieces) * piece, np.arange(1, pieces) * piece - 1, V - 1]
        ids[rng.choice(60000, size=len(edges), replace=False)] = edges
        ids[T - 1] = V - 2
    lse = _check_loss(nt, x, x64, W, W64, ids, 1.0, dtype)
    g_nll, _, g_x, g_W = _check_gradients(nt, x, x64, W, W64, ids, lse, dtype, rng, both=True,
                                          accumulate=True)
    a = nt.nt_token_loss_backward(x, W, _ids(ids), lse, g_nll)
    alone = (nt.nt_token_loss_backward(x, W, _ids(ids), lse, g_nll, weight_grad=False)[0],
             nt.nt_token_loss_backward(x, W, _ids(ids), lse, g_nll, x_grad=False)[1])
    for p, q in zip(a, alone):
        np.testing.assert_array_equal(bits(p, torch), bits(q, torch))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,C", [(1, 300, 64), (33, 130, 8), (257, 128, 1032), (90, 3000, 64)])
def test_loss_gradient_of_the_weights_alone(nt, T, V, C, dtype):
    """Without g_x the weights' gradient has the same bits, added or not."""
    announce(f"loss backward without g_x T={T} V={V} C={C} {dtype}")
    rng = np.random.default_rng(T)
    x, x64, W, W64, ids = _loss_inputs(rng, T, V, C, dtype)
    lse = nt.nt_token_loss(x, W, _ids(ids))[1]
    g = torch.randn(T, device="cuda")
    for old in (None, torch.randn((V, C), device="cuda")):
        a, b = (None, None) if old is None else (old.clone(), old.clone())
        more = old is not None
        _, want = nt.nt_token_loss_backward(x, W, _ids(ids), lse, g, g_W=a, accumulate=more)
        none, got = nt.nt_token_loss_backward(x, W, _ids(ids), lse, g, g_W=b, accumulate=more,
                                              x_grad=False)
        assert none is None
        np.testing.assert_array_equal(bits(got, torch), bits(want, torch))
    for refused in (dict(x_grad=False, weight_grad=False), dict(x_grad=False, g_x=torch.empty_like(x))):
        with pytest.raises(ValueError):
            nt.nt_token_loss_backward(x, W, _ids(ids), lse, g, **refused)


# ---------------------------------------------------------------------- norm
@pytest.mark.parametrize("group", [0, 64])
def test_residual_norm_8bit_smallest_scales(nt, group):
    """Finite values have finite codes where the scale is a few of fp32's smallest steps and
    its rounding leaves quotients past 448: those are 448."""
    step, C = 2.0 ** -149, 128
    tops = [1, 100, 224, 225, 464, 465, 500, 650, 671, 672, 1100, 2000, 5900, 6100, 7000, 10 ** 5]
    rng = np.random.default_rng(6)
    units = np.stack([np.r_[t, -t, 0, rng.integers(-t, t + 1, size=C - 3)] for t in tops])
    units[:, 64:66] = units[:, :2]  # the largest one in every group
    y = (units * step).astype(np.float32)
    assert (y.astype(np.float64) == units * step).all()
    x = torch.from_numpy(y).cuda()
    # the squares are zeros in fp32, so eps = 1 leaves x as it is
    codes, scales, _ = nt.nt_residual_norm_8bit(x, eps=1.0, group=group)
    want = (np.abs(y).max(1) * np.float32(1.0 / 448.0))[:, None]
    s = scales.cpu().numpy()
    np.testing.assert_array_equal(s, np.broadcast_to(want, s.shape))
    got = codes.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    s = s[:, :1].astype(np.float64)
    off = np.abs(got * s - y)
    bound = np.maximum(tb.E4M3_HALF * np.abs(y), tb.E4M3_LEAST_HALF * s)
    # the quotient is off by 2^-22 of it at most, and what is past 448 is lost
    bound = bound + 2.0 ** -22 * np.abs(y) + np.maximum(np.abs(y) - 448 * s, 0.0)
    assert (off <= bound).all()
    x[3, 5], x[8, 70] = math.nan, math.inf
    codes = nt.nt_residual_norm_8bit(x, eps=1.0, group=group)[0].float()
    assert bool(torch.isnan(codes[3]).all())  # the row's mean of squares
    assert bool(torch.isnan(codes[8, 70])) and bool((codes[8, :70] == 0).all())
