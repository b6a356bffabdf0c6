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


# ------------------------------------------------- workspaces, graphs, streams
def _sorted_step(nt, table, tokens, few, w, out, workspaces=(None, None, None)):
    """The operators in the forms that keep state in a workspace: the embedding's gradient by
    sorted tokens, the loss of few tokens, the norm's weights."""
    T, (V, C) = tokens.shape[0], table.shape
    assert nt.nt_token_embedding_backward_workspace_bytes(T, V, C) > 0  # sorted, not direct
    assert few.shape[0] <= 32
    s0 = nt.nt_token_embedding(table, tokens.clamp(max=V - 1), scale=2.0)
    y, h = nt.nt_residual_norm(s0, w, residual=s0)
    nll, lse = nt.nt_token_loss(y[:few.shape[0]], table, few, workspace=workspaces[0])
    g, g_w = nt.nt_residual_norm_backward(h, y, w, workspace=workspaces[1])
    g_table = nt.nt_token_embedding_backward(tokens, g, V, g_table=out, workspace=workspaces[2])
    more = nt.nt_token_embedding_backward(tokens, y, V, g_table=g_table.clone(), accumulate=True,
                                          workspace=workspaces[2])
    return nll, lse, g_w, g_table, more


def _sorted_inputs(dtype, V, C, T, n):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    table = (torch.randn((V, C), device="cuda") * 0.3).to(dt)
    w = torch.ones(C, device="cuda")
    return table, w, _tokens_of(V, T), torch.randint(-1, V, (n,), device="cuda", dtype=torch.int32)


def _tokens_of(V, T):
    """Frequent, rare and absent tokens, and some that the table does not hold."""
    ids = torch.randint(-3, V, (T,), device="cuda", dtype=torch.int32)
    ids[::3] = V // 2
    ids[1::7] = V + 5
    return ids


def _same_bits(got, want):
    for a, b in zip(got, want):
        np.testing.assert_array_equal(bits(a, torch), bits(b, torch))


SORTED = [(6000, 136, 700, 20), (9, 64, 5000, 16), (70001, 24, 4500, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,C,T,n", SORTED)
def test_sorted_and_few_captured_and_replayed(nt, V, C, T, n, dtype):
    """Replays on new inputs, with eager calls and synchronizations between, as eager calls."""
    announce(f"captured V={V} C={C} T={T} {dtype}")
    torch.manual_seed(V)
    table, w, tokens, few = _sorted_inputs(dtype, V, C, T, n)
    out = torch.empty((V, C), device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(2):
            _sorted_step(nt, table, tokens, few, w, out)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _sorted_step(nt, table, tokens, few, w, out)
    for k in range(4):
        tokens.copy_(_tokens_of(V, T) if k % 2 else torch.full_like(tokens, k - 2))
        few.copy_(torch.randint(-1, V, (n,), device="cuda", dtype=torch.int32))
        table.copy_(torch.randn((V, C), device="cuda") * 0.3)
        graph.replay()
        torch.cuda.synchronize()
        held = [t.clone() for t in got]
        _same_bits(held, _sorted_step(nt, table, tokens, few, w, torch.empty_like(out)))


def test_sorted_and_few_on_two_streams(nt):
    """Two streams at once, each call with a workspace of its own."""
    torch.manual_seed(3)
    V, C, T, n = 6000, 136, 3000, 32
    table, w, _, _ = _sorted_inputs("bf16", V, C, T, n)
    batches = [_sorted_inputs("bf16", V, C, T, n)[2:] for _ in range(2)]
    want = [_sorted_step(nt, table, *b, w, None) for b in batches]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in batches], []
    for b, s in zip(batches, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([_sorted_step(nt, table, *b, w, None) for _ in range(5)][-1])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        _same_bits(a, b)


def test_workspaces_shared_by_graphs_and_sizes(nt):
    """One workspace for calls of different sizes in turn, eager ones and two graphs that hold
    it, on one stream: nothing that another call left in it is taken for its own."""
    torch.manual_seed(4)
    cases = [_sorted_inputs("bf16", 6000, 136, 3000, 32), _sorted_inputs("f32", 9, 64, 5000, 7)]
    # torch's allocations are 512 bytes apart, so any size is aligned
    ws = [torch.empty(1 << 24, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(3)]
    step = lambda c: _sorted_step(nt, c[0], c[2], c[3], c[1], None, ws)  # noqa: E731
    want = [[t.clone() for t in _sorted_step(nt, c[0], c[2], c[3], c[1], None)] for c in cases]
    graphs = []
    for c in cases:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step(c)
        torch.cuda.current_stream().wait_stream(stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(c)
        graphs.append((graph, got))
    for k in range(4):
        for c, (graph, got), ref in zip(cases, graphs, want):
            graph.replay()
            held = [t.clone() for t in got]
            torch.cuda.synchronize()
            _same_bits(held, ref)
            if k % 2:
                _same_bits(step(c), ref)
            if k == 2:
                for t in ws:
                    t.fill_(255)


def test_loss_workspace_of_sizes_in_turn(nt):
    """The loss and its gradient in one workspace after larger and smaller calls, and after
    NaN in all of it."""
    rng = np.random.default_rng(2)
    sizes = [(700, 1301, 128, "bf16"), (33, 300, 64, "bf16"), (20, 1000, 64, "f32"),
             (257, 128, 72, "f32"), (300, 900, 200, "bf16")]
    need = max(nt.nt_token_loss_backward_workspace_bytes(*s) for s in sizes)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    for T, V, C, dtype in sizes * 2:
        x, _, W, _, ids = _loss_inputs(rng, T, V, C, dtype)
        g = torch.randn(T, device="cuda")
        a = nt.nt_token_loss(x, W, _ids(ids))
        b = nt.nt_token_loss(x, W, _ids(ids), workspace=ws)
        _same_bits(b, a)
        _same_bits(nt.nt_token_loss_backward(x, W, _ids(ids), a[1], g, workspace=ws),
                   nt.nt_token_loss_backward(x, W, _ids(ids), a[1], g))
