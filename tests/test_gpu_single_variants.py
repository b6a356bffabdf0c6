"""GPU parity of the attention kernels' variants, chosen by what selects them:
type, padded width, tiles that are whole, the number of workgroups. Forward and
gradient against the float64 oracle within the bounds of tests/single_bounds.py,
and each twice, bit by bit."""
import numpy as np
import pytest

import oracle
import single_bounds as sb
from gpu_util import announce, bits, f64
from test_gpu_single import _attention_inputs, _dev, _part, _within, nt  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _check(nt, case, seed, gradient=True):  # noqa: F811
    rows, cols, H, K, D, kind, causal, dtype, layout = case
    rng = np.random.default_rng(seed)
    c, (q, k, v, b), (q64, k64, v64, b64), scale = _attention_inputs(rng, case)
    g, g64 = _dev(rng.normal(size=tuple(q.shape)), dtype)
    p = _part(nt, rows, cols)
    o, lse = nt.nt_single_attention(p, q, k, v, bias=b, causal=causal)
    o2, lse2 = nt.nt_single_attention(p, q, k, v, bias=b, causal=causal)
    torch.cuda.synchronize()
    ro, rl = oracle.attention(rows, c, q64, k64, v64, b64, causal, scale)
    bo, bl = sb.attention_bound(rows, c, q64, k64, v64, ro, rl, b64, causal, scale, dtype)
    o64, l64 = f64(o, torch), f64(lse, torch)
    _within("o", o64, ro, bo)
    _within("lse", l64, rl, bl)
    np.testing.assert_array_equal(bits(o, torch), bits(o2, torch))
    np.testing.assert_array_equal(bits(lse, torch), bits(lse2, torch))
    if not gradient:
        return
    got = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=b, causal=causal)
    again = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=b, causal=causal)
    torch.cuda.synchronize()
    ref = oracle.attention_backward(rows, c, q64, k64, v64, o64, l64, g64, b64, causal, scale)
    bound = sb.attention_backward_bound(rows, c, q64, k64, v64, o64, l64, g64, ref[:3], b64,
                                        causal, scale, dtype)
    for name, x, y, r, e in zip(("g_q", "g_k", "g_v", "g_bias"), got, again, ref, bound):
        if r is not None:
            _within(name, f64(x, torch), r, e)
            np.testing.assert_array_equal(bits(x, torch), bits(y, torch))


WHOLE = [
    # rows, cols, heads, kv_heads, dim, bias, causal, dtype, layout: heads as wide as their
    # padded width, the last sample ending on a whole tile, at the end of its array
    ([64], None, 1, 1, 96, "none", False, "bf16", "split"),
    ([30, 128], None, 2, 2, 96, "none", True, "bf16", "split"),
    ([128, 64], None, 4, 2, 96, "plain", False, "bf16", "split"),
    ([192], None, 2, 1, 96, "masked", True, "bf16", "split"),
    ([1, 2], [100, 640], 4, 2, 96, "none", False, "bf16", "split"),
    ([256], [64], 2, 2, 96, "plain", False, "bf16", "split"),
    ([128], None, 2, 1, 64, "none", False, "bf16", "split"),
    ([128], None, 2, 2, 128, "plain", True, "bf16", "split"),
]


@pytest.mark.parametrize("case", WHOLE)
def test_attention_whole_tiles(nt, case):  # noqa: F811
    announce(f"attention, whole tiles {case}")
    _check(nt, case, 51)


WIDE_F32 = [
    # the fp32 kernels above 64 dimensions, whose tile addresses pass through vector registers;
    # whole tiles and partial ones
    ([64, 128], None, 2, 2, 96, "none", False, "f32", "split"),
    ([70, 33], None, 2, 1, 96, "none", True, "f32", "fused"),
    ([100], None, 4, 2, 88, "none", False, "f32", "split"),
    ([128, 65], None, 2, 2, 128, "none", True, "f32", "split"),
    ([90], None, 2, 1, 104, "none", False, "f32", "split"),
    ([64, 61], None, 2, 2, 96, "plain", False, "f32", "split"),
    ([3], [200], 2, 1, 96, "masked", True, "f32", "split"),
]


@pytest.mark.parametrize("case", WIDE_F32)
def test_attention_wide_f32(nt, case):  # noqa: F811
    announce(f"attention, wide fp32 {case}")
    _check(nt, case, 52)


# What selects a kernel beside its type, its padded width, a bias and the causal bound:
# "many" workgroups (tiles of 128 rows in the forward, without a bias; both walks of the
# gradient on their own, over 128 rows and keys), "some" (on their own, over 64), "few" (both
# walks in one launch), "shared" key heads (on their own, waves that share keys).
RAGGED = [1, 2, 1, 3, 1, 1, 4, 1, 2, 1, 1, 5, 1, 1, 1, 2, 1, 1, 3, 1, 1, 1, 2, 1, 1, 1, 6, 1, 1, 1]
GRIDS = {
    "many": (RAGGED + [140, 70], 64, 64),
    "some": (RAGGED + [140, 70], 50, 50),
    "few": ([70, 0, 129], 2, 2),
    "shared": ([33, 130, 1], 6, 2),
}


def _grid_cases():
    for grid in GRIDS:
        for dtype in ("bf16", "f32"):
            for dim in (32, 64, 96, 128):
                for kind in ("none", "plain"):
                    for causal in (False, True):
                        if grid == "some" and (dtype == "f32" or kind != "none" or not causal):
                            continue  # the same kernels as "many"
                        yield grid, dtype, dim, kind, causal


@pytest.mark.parametrize("grid,dtype,dim,kind,causal", _grid_cases())
def test_attention_kernel(nt, grid, dtype, dim, kind, causal):  # noqa: F811
    """Every second width is eight short of its padded one. The causal bound is a
    constant of the forward's kernels only, so the gradient of many workgroups runs
    with it alone."""
    announce(f"attention kernel {grid} {dtype} {dim} {kind} {causal}")
    lens, H, K = GRIDS[grid]
    D = dim - 8 if causal else dim
    case = (lens, None, H, K, D, kind, causal, dtype, "split")
    _check(nt, case, 53, gradient=causal or grid != "many")
