"""GPU parity of the single attention operators (nt_rotary_table,
nt_qk_norm_rotary and its gradient, nt_single_attention and its gradient) and
of nt_adamw_step against the float64 oracle, element by element within the
bounds that tests/single_bounds.py derives from the arithmetic."""
import math

import numpy as np
import pytest

import oracle
import single_bounds as sb
from gpu_util import announce, bits, f64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": "bfloat16", "f32": "float32"}


@pytest.fixture(scope="module", autouse=True)
def nt():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import padding_free_pair_amd as nt
    nt._native.lib()  # raises if the library is missing: no fallback
    return nt


def _dev(a, dtype="f32"):
    """A device tensor of `dtype` and the float64 values it holds."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(getattr(torch, DT[dtype]))
    return t.cuda(), f64(t, torch)


def _within(name, got, ref, bound):
    """Every element within its bound; NaN and infinities in the same places."""
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = np.isfinite(ref)
    np.testing.assert_array_equal(got[~fine], ref[~fine], err_msg=name)
    assert np.isfinite(got[fine]).all(), name
    off = np.abs(got - np.where(fine, ref, 0.0))
    over = fine & (off > bound)
    assert not over.any(), (name, int(over.sum()), float((off[fine] / np.broadcast_to(
        bound, off.shape)[fine]).max()))


def _fused(rng, T, H, K, D, dtype):
    x, x64 = _dev(rng.normal(size=(T, H + 2 * K, D)), dtype)
    cut = [slice(0, H), slice(H, H + K), slice(H + K, H + 2 * K)]
    return [x[:, c] for c in cut], [x64[:, c] for c in cut]


def _part(nt, rows, cols=None):
    return nt.nt_make_partition(rows) if cols is None else nt.nt_make_partition_rect(rows, cols)


# --------------------------------------------------------------------- table
@pytest.mark.parametrize("kw", [
    {}, {"base": 500000.0}, {"scaling": "linear", "factor": 8.0},
    {"scaling": "parts", "factor": 4.0, "original": 2048.0, "magnitude": 1.1386},
    {"scaling": "parts", "factor": 32.0, "original": 8192.0, "beta_fast": 4.0, "beta_slow": 0.5}])
def test_rotary_table(nt, kw):
    for positions, R in ((1, 2), (37, 24), (3000, 64)):
        announce(f"rotary table {positions} x {R} {kw}")
        got = f64(nt.nt_rotary_table(positions, R, **kw), torch)
        # one rounding; the fp64 angle (up to 3,000) is off by a few 2^-53 of itself
        _within("table", got, oracle.rotary_table(positions, R, **kw), 2.0 ** -24 * 1.2 + 1e-11)


def test_rotary_table_far(nt):
    """Positions past 10^6, where a 32-bit angle would be off by 0.03."""
    announce("rotary table to 2^20 + 5")
    n = (1 << 20) + 5
    t = nt.nt_rotary_table(n, 8)
    at = np.array([n - 1, n - 2, 1 << 20, 777_777])
    ref = np.concatenate([f(at[:, None] * oracle.rotary_frequencies(8)[None])
                          for f in (np.cos, np.sin)], 1)
    got = f64(t[torch.from_numpy(at).cuda()], torch)
    _within("table", got, ref, 2.0 ** -24 + 1e-9)


# ---------------------------------------------------------------------- norm
NORMS = [
    # lengths, heads, kv_heads, dim, rot, interleaved, dtype, layout
    ([7, 0, 33, 1], 4, 4, 32, 32, False, "bf16", "split"),
    ([7, 0, 33, 1], 4, 2, 32, 32, False, "f32", "fused"),
    ([100], 3, 1, 24, 24, False, "bf16", "split"),        # half of the rotated part is 12
    ([5, 6], 2, 2, 40, 10, False, "f32", "split"),        # rotated part ends inside a lane
    ([64, 3], 5, 1, 128, 64, True, "bf16", "fused"),
    ([1], 1, 1, 8, 8, True, "f32", "split"),
    ([31, 2], 2, 1, 128, 128, False, "bf16", "fused"),
    ([31, 2], 2, 0, 64, 2, False, "bf16", "split"),       # queries alone
    ([600, 1200], 16, 4, 64, 48, False, "f32", "split"),  # several workgroups of partial sums
    ([9, 4], 2, 2, 16, 0, False, "bf16", "split"),        # norm alone
]


def _norm_inputs(rng, case):
    lens, H, K, D, R, inter, dtype, layout = case
    T = sum(lens)
    if layout == "fused":
        (q, k, _), (q64, k64, _) = _fused(rng, T, H, K, D, dtype)
    else:
        q, q64 = _dev(rng.normal(size=(T, H, D)), dtype)
        k, k64 = _dev(rng.normal(size=(T, K, D)), dtype) if K else (None, None)
    return q, q64, k, k64


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("case", NORMS)
def test_norm_rotary(nt, case, norm):
    lens, H, K, D, R, inter, dtype, layout = case
    announce(f"norm rotary {case} norm={norm}")
    rng = np.random.default_rng(11)
    q, q64, k, k64 = _norm_inputs(rng, case)
    w, w64 = _dev(1 + 0.2 * rng.normal(size=(2, D)))
    ws, w64 = ((w[0], w[1].contiguous()), w64) if norm else ((None, None), (None, None))
    table = nt.nt_rotary_table(max(lens), R) if R else None
    t64 = f64(table, torch) if R else None
    p = _part(nt, lens)
    out = nt.nt_qk_norm_rotary(p, q, k, ws[0], ws[1], table, interleaved=inter)
    torch.cuda.synchronize()
    for x64, wx, got in ((q64, w64[0], out[0]), (k64, w64[1], out[1])):
        if x64 is None:
            assert got is None
            continue
        ref = oracle.norm_rotary(x64, wx, t64, oracle.positions_of(lens), inter)
        _within("norm", f64(got, torch), ref, sb.norm_bound(x64, wx, ref, t64, dtype))


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("case", NORMS)
def test_norm_rotary_backward(nt, case, norm):
    lens, H, K, D, R, inter, dtype, layout = case
    announce(f"norm rotary backward {case} norm={norm}")
    rng = np.random.default_rng(12)
    q, q64, k, k64 = _norm_inputs(rng, case)
    w, w64 = _dev(1 + 0.2 * rng.normal(size=(2, D)))
    ws, w64 = ((w[0], w[1].contiguous()), w64) if norm else ((None, None), (None, None))
    T = sum(lens)
    g, g64 = zip(*[_dev(rng.normal(size=(T, h, D)), dtype) if h else (None, None) for h in (H, K)])
    table = nt.nt_rotary_table(max(lens), R) if R else None
    t64 = f64(table, torch) if R else None
    p = _part(nt, lens)
    call = lambda: nt.nt_qk_norm_rotary_backward(p, q, k, g[0], g[1], ws[0], ws[1],  # noqa: E731
                                                 table, interleaved=inter)
    got, again = call(), call()
    torch.cuda.synchronize()
    for i, x64 in enumerate((q64, k64)):
        if x64 is None:
            assert got[i] is None
            continue
        rx, rw = oracle.norm_rotary_backward(x64, g64[i], w64[i], t64, oracle.positions_of(lens),
                                             inter)
        bx, bw = sb.norm_backward_bound(x64, w64[i], g64[i], rx, dtype)
        _within("g_x", f64(got[i], torch), rx, bx)
        np.testing.assert_array_equal(bits(got[i], torch), bits(again[i], torch))
        if norm:
            _within("g_w", f64(got[2 + i], torch), rw, bw)
            np.testing.assert_array_equal(bits(got[2 + i], torch), bits(again[2 + i], torch))
        else:
            assert got[2 + i] is None


def test_norm_rotary_positions_and_in_place(nt):
    """Given positions (one outside the table: NaN), in place within a fused
    array whose third part stays as it was."""
    announce("norm rotary positions, in place")
    rng = np.random.default_rng(13)
    lens, H, K, D = [5, 9], 4, 2, 64
    x, x64 = _dev(rng.normal(size=(14, H + 2 * K, D)), "bf16")
    w, w64 = _dev(1 + 0.1 * rng.normal(size=(D,)))
    at = rng.integers(0, 50, 14)
    pos = torch.from_numpy(at.astype(np.int32)).cuda()
    bad = pos.clone()
    bad[3], bad[7] = 50, -1
    table = nt.nt_rotary_table(50, D)
    p = _part(nt, lens)
    q, k = x[:, :H], x[:, H:H + K]
    out = nt.nt_qk_norm_rotary(p, q, k, w, w, table, positions_q=bad, positions_k=pos,
                               q_out=q, k_out=k)
    assert out[0].data_ptr() == q.data_ptr()
    got = f64(x, torch)
    ref = oracle.norm_rotary(x64, w64, f64(table, torch), at)
    bound = sb.norm_bound(x64, w64, ref, f64(table, torch), "bf16")
    keep = [i for i in range(14) if i not in (3, 7)]
    assert np.isnan(got[[3, 7], :H]).all()
    _within("q", got[keep, :H], ref[keep, :H], bound[keep, :H])
    _within("k", got[:, H:H + K], ref[:, H:H + K], bound[:, H:H + K])
    np.testing.assert_array_equal(got[:, H + K:], x64[:, H + K:])


def test_norm_rotary_rectangular(nt):
    """Keys belong to the columns of a rectangular partition."""
    announce("norm rotary rectangular")
    rng = np.random.default_rng(14)
    rows, cols = [3, 0, 1, 5], [8, 4, 0, 40]
    q, q64 = _dev(rng.normal(size=(9, 2, 32)), "bf16")
    k, k64 = _dev(rng.normal(size=(52, 2, 32)), "bf16")
    w, w64 = _dev(np.ones(32))
    table = nt.nt_rotary_table(40, 32)
    out = nt.nt_qk_norm_rotary(_part(nt, rows, cols), q, k, w, w, table)
    for x64, lens, got in ((q64, rows, out[0]), (k64, cols, out[1])):
        ref = oracle.norm_rotary(x64, w64, f64(table, torch), oracle.positions_of(lens))
        _within("out", f64(got, torch), ref, sb.norm_bound(x64, w64, ref, 1, "bf16"))


# ----------------------------------------------------------------- attention
ATTENTIONS = [
    # rows, cols, heads, kv_heads, dim, bias, causal, dtype, layout
    ([7, 12, 5, 16], None, 2, 2, 8, "plain", False, "f32", "split"),
    ([1], None, 1, 1, 8, "none", True, "bf16", "split"),
    ([33, 0, 64, 1, 130], None, 4, 2, 32, "masked", False, "bf16", "fused"),
    ([33, 0, 64, 1, 130], None, 4, 1, 40, "masked", True, "f32", "split"),
    ([257, 129], None, 6, 3, 64, "none", True, "bf16", "fused"),
    ([300], None, 2, 2, 96, "plain", True, "bf16", "split"),
    ([200, 63], None, 3, 1, 128, "none", False, "f32", "fused"),
    ([190, 61], None, 4, 1, 128, "plain", False, "bf16", "split"),
    ([65] * 20, None, 2, 2, 24, "plain", False, "bf16", "split"),
    ([3] * 300, None, 2, 1, 16, "none", False, "bf16", "split"),   # samples beyond one search step
    # queries over other columns; single tokens; no columns at all; more rows than columns
    ([1, 1, 1, 1], [700, 33, 0, 1], 8, 2, 128, "none", False, "bf16", "split"),
    ([1, 2, 3], [1500, 64, 65], 4, 4, 64, "plain", False, "f32", "split"),
    ([5, 40, 0, 9], [40, 5, 7, 0], 2, 1, 48, "masked", True, "bf16", "split"),
    ([2, 1], [1100, 900], 5, 1, 72, "masked", True, "bf16", "split"),
    ([20, 150], [150, 20], 2, 2, 32, "none", True, "f32", "split"),
]


def _attention_inputs(rng, case):
    rows, cols, H, K, D, kind, causal, dtype, layout = case
    c = cols or rows
    T, Tc = sum(rows), sum(c)
    if layout == "fused":
        (q, k, v), (q64, k64, v64) = _fused(rng, T, H, K, D, dtype)
    else:
        (q, q64), (k, k64), (v, v64) = (_dev(rng.normal(size=s), dtype) for s in (
            (T, H, D), (Tc, K, D), (Tc, K, D)))
    cells = sum(n * m for n, m in zip(rows, c))
    bias = bias64 = None
    if kind != "none":
        b = rng.normal(size=(H, cells)) * 2
        if kind == "masked":
            b[:, rng.random(cells) < 0.2] = -np.inf
            at = 0
            for n, m in zip(rows, c):  # the middle row of every sample sees nothing
                b[:, at + n // 2 * m:at + (n // 2 + 1) * m if n else at] = -np.inf
                at += n * m
        bias, bias64 = _dev(b, dtype)
    return c, (q, k, v, bias), (q64, k64, v64, bias64), 1 / math.sqrt(D)


@pytest.mark.parametrize("case", ATTENTIONS)
def test_attention(nt, case):
    rows, cols, H, K, D, kind, causal, dtype, layout = case
    announce(f"attention {case}"[:300])
    c, (q, k, v, b), (q64, k64, v64, b64), scale = _attention_inputs(np.random.default_rng(21), case)
    p = _part(nt, rows, cols)
    o, lse = nt.nt_single_attention(p, q, k, v, bias=b, causal=causal)
    o2, lse2 = nt.nt_single_attention(p, q, k, v, bias=b, causal=causal)
    torch.cuda.synchronize()
    ro, rl = oracle.attention(rows, c, q64, k64, v64, b64, causal, scale)
    bo, bl = sb.attention_bound(rows, c, q64, k64, v64, ro, rl, b64, causal, scale, dtype)
    _within("o", f64(o, torch), ro, bo)
    _within("lse", f64(lse, torch), rl, bl)
    np.testing.assert_array_equal(bits(o, torch), bits(o2, torch))
    np.testing.assert_array_equal(bits(lse, torch), bits(lse2, torch))


@pytest.mark.parametrize("case", ATTENTIONS)
def test_attention_backward(nt, case):
    rows, cols, H, K, D, kind, causal, dtype, layout = case
    announce(f"attention backward {case}"[:300])
    rng = np.random.default_rng(22)
    c, (q, k, v, b), (q64, k64, v64, b64), scale = _attention_inputs(rng, case)
    g, g64 = _dev(rng.normal(size=tuple(q.shape)), dtype)
    p = _part(nt, rows, cols)
    ro, rl = oracle.attention(rows, c, q64, k64, v64, b64, causal, scale)
    o, o64 = _dev(ro, dtype)
    lse, l64 = _dev(rl)
    call = lambda: nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=b,  # noqa: E731
                                                   causal=causal)
    got, again = call(), call()
    torch.cuda.synchronize()
    ref = oracle.attention_backward(rows, c, q64, k64, v64, o64, l64, g64, b64, causal, scale)
    bound = sb.attention_backward_bound(rows, c, q64, k64, v64, o64, l64, g64, ref[:3], b64,
                                        causal, scale, dtype)
    for name, x, y, r, e in zip(("g_q", "g_k", "g_v", "g_bias"), got, again, ref, bound):
        if r is None:
            assert x is None
            continue
        _within(name, f64(x, torch), r, e)
        np.testing.assert_array_equal(bits(x, torch), bits(y, torch))


SPLITS = [
    # few rows (parts of equal length, most of them empty in short samples), then many rows
    ([1, 1, 0, 2, 1, 1], [5000, 1, 700, 0, 64, 3001], 8, 2, 128, "none", False, "bf16", "split"),
    ([1, 2, 1], [2500, 65, 129], 4, 2, 64, "masked", True, "bf16", "split"),
    ([1] * 4, [3000, 900, 513, 300], 2, 1, 40, "plain", False, "f32", "split"),
    ([1] * 70, [8] * 69 + [50000], 4, 4, 32, "none", False, "bf16", "split"),
    ([150, 3], [2100, 40], 2, 1, 64, "masked", True, "f32", "split"),
]


@pytest.mark.parametrize("case", SPLITS)
def test_attention_split_over_keys(nt, case):
    """Parts behind a row's last key leave nothing: the workspace holds NaN before."""
    rows, cols, H, K, D, kind, causal, dtype, layout = case
    announce(f"attention split {case}"[:300])
    c, (q, k, v, b), (q64, k64, v64, b64), scale = _attention_inputs(np.random.default_rng(23), case)
    p = _part(nt, rows, cols)
    need = nt.nt_attention_workspace_bytes(p, H, K, D, q.dtype, causal)
    assert need > 0
    ws = torch.full((need // 4,), float("nan"), dtype=torch.float32, device="cuda")
    o, lse = nt.nt_single_attention(p, q, k, v, bias=b, causal=causal, workspace=ws)
    torch.cuda.synchronize()
    ro, rl = oracle.attention(rows, c, q64, k64, v64, b64, causal, scale)
    bo, bl = sb.attention_bound(rows, c, q64, k64, v64, ro, rl, b64, causal, scale, dtype)
    _within("o", f64(o, torch), ro, bo)
    _within("lse", f64(lse, torch), rl, bl)


MANY = [
    # enough workgroups for tiles of 128 rows, for two launches of the gradient, and wide heads
    ([32] * 256 + [0, 45, 1, 90], None, 8, 8, 16, "none", True, "bf16", "fused"),
    ([64] * 139 + [30], None, 8, 8, 24, "masked", False, "bf16", "split"),
    ([64] * 139 + [30], None, 8, 4, 32, "none", False, "f32", "split"),
    ([64] * 40, None, 8, 8, 128, "plain", True, "bf16", "split"),
    ([64] * 40, None, 16, 8, 72, "none", False, "bf16", "fused"),
    ([50, 70], None, 2, 2, 128, "plain", True, "f32", "split"),
]


@pytest.mark.parametrize("case", MANY)
def test_attention_many_workgroups(nt, case):
    rows, cols, H, K, D, kind, causal, dtype, layout = case
    announce(f"attention, many workgroups {case[2:]}")
    rng = np.random.default_rng(24)
    c, (q, k, v, b), (q64, k64, v64, b64), scale = _attention_inputs(rng, case)
    g, g64 = _dev(rng.normal(size=tuple(q.shape)), dtype)
    p = _part(nt, rows, cols)
    o, lse = nt.nt_single_attention(p, q, k, v, bias=b, causal=causal)
    got = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=b, causal=causal)
    again = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=b, causal=causal)
    torch.cuda.synchronize()
    ro, rl = oracle.attention(rows, c, q64, k64, v64, b64, causal, scale)
    bo, bl = sb.attention_bound(rows, c, q64, k64, v64, ro, rl, b64, causal, scale, dtype)
    o64, l64 = f64(o, torch), f64(lse, torch)
    _within("o", o64, ro, bo)
    _within("lse", l64, rl, bl)
    ref = oracle.attention_backward(rows, c, q64, k64, v64, o64, l64, g64, b64, causal, scale)
    bound = sb.attention_backward_bound(rows, c, q64, k64, v64, o64, l64, g64, ref[:3], b64,
                                        causal, scale, dtype)
    for name, x, y, r, e in zip(("g_q", "g_k", "g_v", "g_bias"), got, again, ref, bound):
        if r is not None:
            _within(name, f64(x, torch), r, e)
            np.testing.assert_array_equal(bits(x, torch), bits(y, torch))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_lowest_value_masks(nt, dtype):
    """A bias of the type's lowest value leaves a row's other keys, and a row
    that holds nothing else weighs its keys alike (the scores vanish beside
    it); NaN and infinities past the causal bound are not read."""
    announce(f"attention lowest masks {dtype}")
    rng = np.random.default_rng(23)
    n, H, D = 70, 2, 32
    low = float(torch.finfo(getattr(torch, DT[dtype])).min)
    b = rng.normal(size=(H, n, n))
    b[:, :, ::3] = low
    b[:, 5] = low
    b[:, np.triu_indices(n, 1)[0], np.triu_indices(n, 1)[1]] = np.nan
    b[:, 2, 40:] = np.inf
    b[:, 0, 0] = low
    (q, q64), (k, k64), (v, v64) = (_dev(rng.normal(size=(n, H, D)), dtype) for _ in range(3))
    bias, b64 = _dev(b.reshape(H, -1), dtype)
    p = _part(nt, [n])
    scale = 1 / math.sqrt(D)
    o, lse = nt.nt_single_attention(p, q, k, v, bias=bias, causal=True)
    seen = np.tril(np.ones((n, n), bool)).reshape(-1)
    clean = np.where(seen, np.where(b64 < -1e38, -1e30, b64), 0.0)  # the same weights
    ro, rl = oracle.attention([n], [n], q64, k64, v64, clean, True, scale)
    rows = np.r_[0, 1:5, 6:n]
    got, gl = f64(o, torch), f64(lse, torch)
    small = np.where(clean < -1e29, -np.inf, clean)  # such keys weigh nothing beside others
    bo, bl = sb.attention_bound([n], [n], q64, k64, v64, ro, rl, small, True, scale, dtype)
    _within("o", got[rows], ro[rows], bo[rows])
    _within("lse", gl[rows[1:]], rl[rows[1:]], bl[rows[1:]])
    mean = v64[:6].mean(0)
    _within("row 5", got[5], mean, sb.HALF[dtype] * (np.abs(v64[:6]).mean(0) + np.abs(mean)) + 1e-6)
    assert np.all(gl[[0, 5]] < 0.99 * low) and np.all(np.isfinite(gl[[0, 5]]))
    g, _ = _dev(rng.normal(size=(n, H, D)), dtype)
    grads = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=bias, causal=True)
    gb = f64(grads[3], torch).reshape(H, n, n)
    assert all(np.isfinite(f64(x, torch)).all() for x in grads)
    assert np.all(gb[:, ~np.tril(np.ones((n, n), bool))] == 0)


def test_attention_neighbours_do_not_leak(nt):
    """A sample of NaN between two others changes neither, in either direction
    and both types; guard rows around every output stay as they were."""
    rng = np.random.default_rng(24)
    rows, H, K, D = [37, 30, 75], 2, 1, 64
    for dtype in ("bf16", "f32"):
        announce(f"attention neighbours {dtype}")
        T, cells = sum(rows), sum(n * n for n in rows)
        t = getattr(torch, DT[dtype])

        def make(nan):
            r = np.random.default_rng(25)
            q, k, v, g = (_dev(r.normal(size=(T, h, D)), dtype)[0] for h in (H, K, K, H))
            b = _dev(r.normal(size=(H, cells)), dtype)[0]
            if nan:
                for x in (q, k, v, g):
                    x[37:67] = math.nan
                b[:, 37 * 37:37 * 37 + 900] = math.nan
            return q, k, v, g, b

        outs = []
        p = _part(nt, rows)
        for nan in (False, True):
            q, k, v, g, b = make(nan)
            guard = [torch.full((T + 2, h, D), 7.0, dtype=t, device="cuda") for h in (H, H, K, K)]
            gb = torch.full((H * cells + 64,), 7.0, dtype=t, device="cuda")
            o, gq, gk, gv = (x[1:-1] for x in guard)
            lse = torch.full((T + 16, H), 7.0, device="cuda")
            g_bias = gb[32:-32].view(H, cells)
            nt.nt_single_attention(p, q, k, v, bias=b, o=o, lse=lse[8:-8])
            nt.nt_single_attention_backward(p, q, k, v, o, lse[8:-8], g, bias=b, g_q=gq, g_k=gk,
                                            g_v=gv, g_bias=g_bias)
            torch.cuda.synchronize()
            assert all(bool((x[0] == 7).all() and (x[-1] == 7).all()) for x in guard)
            assert bool((lse[:8] == 7).all() and (lse[-8:] == 7).all())
            assert bool((gb[:32] == 7).all() and (gb[-32:] == 7).all())
            keep = np.r_[0:37, 67:T]
            outs.append([bits(x, torch)[keep] for x in (o, lse[8:-8], gq, gk, gv)] +
                        [bits(g_bias, torch)[:, np.r_[0:1369, 1369 + 900:cells]]])
        for x, y in zip(*outs):
            np.testing.assert_array_equal(x, y)


def test_attention_gradient_against_differences(nt):
    """The fp32 gradient against central differences of the fp32 forward. With a
    step h the forward's rounding (2^-20 of outputs of size 1, summed over
    the output) enters as 1e-6 / h and the third derivative as h^2."""
    announce("attention differences")
    rng = np.random.default_rng(26)
    rows, H, K, D = [6, 9], 2, 1, 16
    T, cells = 15, 36 + 81
    (q, _), (k, _), (v, _), (g, _) = (_dev(rng.normal(size=(T, h, D))) for h in (H, K, K, H))
    b, _ = _dev(rng.normal(size=(H, cells)))
    p = _part(nt, rows)

    def loss(*xs):
        o, _ = nt.nt_single_attention(p, *xs[:3], bias=xs[3], causal=True)
        return float((o.double() * g.double()).sum())

    o, lse = nt.nt_single_attention(p, q, k, v, bias=b, causal=True)
    grads = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=b, causal=True)
    for x, gx in zip((q, k, v, b), grads):
        d = torch.from_numpy(rng.normal(size=tuple(x.shape)).astype(np.float32)).cuda()
        h = 5e-3
        args = [q, k, v, b]
        at = [y is x for y in args].index(True)
        up, down = list(args), list(args)
        up[at], down[at] = x + h * d, x - h * d
        num = (loss(*up) - loss(*down)) / (2 * h)
        ana = float((gx.double() * d.double()).sum())
        size = float((gx.double() * d.double()).abs().sum())
        assert abs(num - ana) <= 5e-3 * size, (at, num, ana)


# -------------------------------------------------------------------- AdamW
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def _adamw_case(nt, sizes, dtype, bits_, master, seed=31):
    rng = np.random.default_rng(seed)
    t = getattr(torch, DT[dtype])
    full = [torch.from_numpy(rng.normal(size=n).astype(np.float32)).cuda() for n in sizes]
    params = [x.to(t, copy=True) for x in full]
    grads = [torch.from_numpy(rng.normal(size=n).astype(np.float32)).cuda() for n in sizes]
    m, v, ms, vs = nt.nt_adamw_states(params, bits_)
    return params, grads, m, v, ms, vs, full if master else None


def _values(codes, scales, n):
    if scales is None:
        return f64(codes, torch)
    c = oracle.e4m3_values()[codes.view(torch.uint8).cpu().numpy()]
    return c * np.repeat(f64(scales, torch), 256)[:n]


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("bits_", [32, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_adamw(nt, dtype, bits_, master):
    """Three steps, each against the oracle from the state that the step
    began with; sizes around a lane's, a block's and a workgroup's edges, and
    more tensors than one launch takes."""
    sizes = [1, 3, 4, 7, 255, 256, 257, 1000, 4095, 4096, 4097, 0, 20011] + [5] * 40
    announce(f"adamw {dtype} {bits_} master={master}")
    params, grads, m, v, ms, vs, masters = _adamw_case(nt, sizes, dtype, bits_, master)
    h = nt.nt_adamw_tensors(params, grads, m, v, ms, vs, masters)
    rng = np.random.default_rng(32)
    for step in (1, 2, 3):
        before = []
        for i, n in enumerate(sizes):
            w = f64(masters[i] if masters else params[i], torch)
            a = _values(m[i], ms and ms[i], n)
            r = _values(v[i], vs and vs[i], n)
            before.append((w, a, r * r if bits_ == 8 else r))
            grads[i].copy_(torch.from_numpy((rng.normal(size=n) * 10.0 ** rng.integers(-6, 3, n))
                                            .astype(np.float32)))
        nt.nt_adamw_step(h, step, **HYPER)
        torch.cuda.synchronize()
        for i, n in enumerate(sizes):
            w0, m0, v0 = before[i]
            g = f64(grads[i], torch)
            w, a, b = oracle.adamw(w0, g, m0, v0, step, **HYPER)
            # m, v: three operations on terms of one sign pattern; the parameter: two
            # statistics with ten operations, the update's terms added
            u = sb.U
            em = 4 * u * (np.abs(m0) + np.abs(g))
            ev = 6 * u * b
            mhat, vhat = np.abs(a) / (1 - 0.9 ** step), b / (1 - 0.99 ** step)
            move = mhat / (np.sqrt(vhat) + 1e-8)
            ew = 4 * u * np.abs(w0) + 1e-2 * (
                24 * u * move + em / (1 - 0.9 ** step) / (np.sqrt(vhat) + 1e-8))
            if masters:
                _within("master", f64(masters[i], torch), w, ew)
                np.testing.assert_array_equal(bits(params[i], torch),
                                              bits(masters[i].to(params[i].dtype), torch))
            else:
                _within("param", f64(params[i], torch), w, ew + sb.HALF[dtype] * np.abs(w))
            if bits_ == 32:
                _within("m", f64(m[i], torch), a, em)
                _within("v", f64(v[i], torch), b, ev)
                continue
            for x, codes, scales, e in ((a, m[i], ms[i], em), (np.sqrt(b), v[i], vs[i], 8 * u * np.sqrt(b))):
                top = oracle.block_scales(x) if n else np.zeros(0)
                _within("scale", f64(scales, torch), top, 6 * u * top + (
                    np.array([e[j:j + 256].max() for j in range(0, n, 256)]) / 448 if n else 0))
                s = np.repeat(top, 256)[:n]
                # half a step of e4m3 is 2^-4 of the value, and 2^-10 of a scale below its
                # normal range; a positive root keeps the least code (2^-9)
                half = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s)
                if codes is v[i]:
                    half = np.where((x > 0) & (x < 2.0 ** -9 * s), 2.0 ** -9 * s, half)
                _within("state", _values(codes, scales, n), x, half * (1 + 1e-4) + 2 * e)
            if n:
                code = v[i].view(torch.uint8)
                assert bool((code[torch.from_numpy(b > 1e-30).cuda()] > 0).all())


def test_adamw_rounds_to_nearest_even(nt):
    """8-bit codes of chosen quotients: exact values keep theirs, ties go to the
    even code, as torch's cast rounds."""
    announce("adamw ties")
    vals = oracle.e4m3_values()[:127]
    mid = (vals[:-1] + vals[1:]) / 2
    x = np.concatenate([[448.0], vals, -vals, mid[1:], -mid[1:]])[:512]
    x = np.concatenate([x[:256], [448.0], x[256:]])
    g = torch.from_numpy(x.astype(np.float32)).cuda()
    w = torch.zeros_like(g)
    m, v, ms, vs = nt.nt_adamw_states([w], 8)
    # beta1 = 0: m is the gradient itself; every block's largest value is 448, its scale 1
    nt.nt_adamw_step(nt.nt_adamw_tensors([w], [g], m, v, ms, vs), 1, lr=0.0, beta1=0.0)
    want = (0.0 + g).to(torch.float8_e4m3fn)  # 0 m + g: a negative zero becomes zero
    np.testing.assert_array_equal(m[0].view(torch.uint8).cpu().numpy(),
                                  want.view(torch.uint8).cpu().numpy())


def test_adamw_not_finite(nt):
    """An infinity or NaN in a gradient marks its own element of an 8-bit state
    and leaves its block's other values and scale."""
    announce("adamw not finite")
    g = torch.ones(600, device="cuda")
    g[5], g[300] = math.inf, math.nan
    w = torch.ones(600, device="cuda")
    m, v, ms, vs = nt.nt_adamw_states([w], 8)
    nt.nt_adamw_step(nt.nt_adamw_tensors([w], [g], m, v, ms, vs), 1)
    torch.cuda.synchronize()
    bad = np.zeros(600, bool)
    bad[[5, 300]] = True
    for c, s in ((m[0], ms[0]), (v[0], vs[0])):
        x = _values(c, s, 600)
        assert np.isnan(x[bad]).all() and np.isfinite(x[~bad]).all()
        assert np.isfinite(f64(s, torch)).all()
    assert np.isfinite(f64(w, torch)[~bad]).all()


# ----------------------------------------------- streams, graphs, one step
def _chain_inputs(seed=41):
    rng = np.random.default_rng(seed)
    lens, H, K, D, c_s = [50, 0, 33, 90], 4, 2, 32, 64
    T, cells = sum(lens), sum(n * n for n in lens)
    s, s64 = _dev(rng.normal(size=(T, c_s)), "bf16")
    W, W64 = _dev(rng.normal(size=((H + 2 * K) * D, c_s)) / 8, "bf16")
    bias, b64 = _dev(rng.normal(size=(H, cells)), "bf16")
    w, w64 = _dev(1 + 0.1 * rng.normal(size=(D,)))
    g, g64 = _dev(rng.normal(size=(T, H, D)), "bf16")
    return lens, (H, K, D), (s, W, bias, w, g), (s64, W64, b64, w64, g64)


def _step(nt, p, dims, dev, table, handle, grad, step):
    """Projection, norm and rotation, attention, their gradients, the weight's
    gradient and its update, as one training step runs them."""
    H, K, D = dims
    s, W, bias, w, g = dev
    T = s.shape[0]
    x = (s.float() @ W.float().t()).to(torch.bfloat16).view(T, H + 2 * K, D)
    q, k, v = x[:, :H], x[:, H:H + K], x[:, H + K:]
    qr, kr = nt.nt_qk_norm_rotary(p, q, k, w, w, table)
    o, lse = nt.nt_single_attention(p, qr, kr, v, bias=bias)
    gx = torch.empty_like(x)
    gq, gk, _, gb = nt.nt_single_attention_backward(p, qr, kr, v, o, lse, g, bias=bias,
                                                    g_v=gx[:, H + K:])
    _, _, gw, _ = nt.nt_qk_norm_rotary_backward(p, q, k, gq, gk, w, w, table, g_q_in=gx[:, :H],
                                                g_k_in=gx[:, H:H + K])
    torch.mm(gx.view(T, -1).float().t().contiguous(), s.float(), out=grad)
    nt.nt_adamw_step(handle, step, lr=1e-2)
    return o, lse, gx, gb, gw


def test_training_step_together(nt):
    """The operators one after another against the oracle composed the same way,
    each fed with what the one before it stored."""
    announce("training step together")
    lens, (H, K, D), dev, ref = _chain_inputs()
    s, W, bias, w, g = dev
    p = _part(nt, lens)
    table = nt.nt_rotary_table(max(lens), D)
    grad = torch.empty(W.shape, dtype=torch.float32, device="cuda")
    before = W.clone()
    master = W.float().clone()
    m, v, _, _ = nt.nt_adamw_states([W])
    handle = nt.nt_adamw_tensors([W], [grad], m, v, masters=[master])
    o, lse, gx, gb, gw = _step(nt, p, (H, K, D), dev, table, handle, grad, 1)
    torch.cuda.synchronize()
    s64, W64, b64, w64, g64 = ref
    t64, at = f64(table, torch), oracle.positions_of(lens)
    x = (s64 @ W64.T).reshape(len(s64), -1, D)
    q, k, v_ = x[:, :H], x[:, H:H + K], x[:, H + K:]
    qr, kr = (oracle.norm_rotary(y, w64, t64, at) for y in (q, k))
    scale = 1 / math.sqrt(D)
    ro, rl = oracle.attention(lens, lens, qr, kr, v_, b64, False, scale)
    rq, rk, rv, rb = oracle.attention_backward(lens, lens, qr, kr, v_, ro, rl, g64, b64, False, scale)
    (hq, hwq), (hk, _) = (oracle.norm_rotary_backward(y, gy, w64, t64, at)
                          for y, gy in ((q, rq), (k, rk)))
    rx = np.concatenate([hq, hk, rv], 1)
    rgrad = rx.reshape(len(s64), -1).T @ s64
    # eight roundings to bf16 follow one another (x, q and k, P, o, dS, the gradients twice,
    # the mean's part): each adds at most 2^-8 of the tensor's size to the norm of the error
    for name, got, want in (("o", o, ro), ("gx", gx, rx), ("gb", gb, rb), ("gw", gw, hwq),
                            ("grad", grad, rgrad)):
        off = np.linalg.norm(f64(got, torch).reshape(want.shape) - want) / np.linalg.norm(want)
        assert off <= 8 * 2.0 ** -8, (name, off)
    wr, _, _ = oracle.adamw(f64(before, torch), f64(grad, torch), 0.0, 0.0, 1, 1e-2, 0.9, 0.999,
                            1e-8, 0.01)
    _within("master", f64(master, torch), wr, 1e-6)
    np.testing.assert_array_equal(bits(W, torch), bits(master.to(torch.bfloat16), torch))


def test_step_captured_and_on_another_stream(nt):
    """The whole step in a graph, replayed with eager steps between; the step's
    number and the rate live on the device. Then eagerly on a second stream."""
    announce("training step captured")
    lens, dims, dev, _ = _chain_inputs(42)
    s, W0, bias, w, g = dev
    H, K, D = dims
    p = _part(nt, lens)
    table = nt.nt_rotary_table(max(lens), D)

    def fresh():
        W = W0.clone()
        grad = torch.zeros(W.shape, dtype=torch.float32, device="cuda")
        m, v, ms, vs = nt.nt_adamw_states([W], 8)
        return W, grad, nt.nt_adamw_tensors([W], [grad], m, v, ms, vs)

    def run(state, step):
        W, grad, handle = state
        return _step(nt, p, dims, (s, W, bias, w, g), table, handle, grad, step)

    eager = fresh()
    want = []
    for i in (1, 2, 3, 4):
        outs = run(eager, i)
        want.append([bits(x, torch) for x in outs] + [bits(eager[0], torch)])
    captured = fresh()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the libraries' own warm-up
        run(fresh(), 1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        outs = run(captured, step)
    torch.cuda.synchronize()
    other = fresh()
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        got = [bits(x, torch) for x in outs] + [bits(captured[0], torch)]
        for a, b in zip(got, want[i]):
            np.testing.assert_array_equal(a, b)
        run(other, i + 1)  # eager work of the program between the replays
        torch.cuda.synchronize()
    announce("training step on another stream")
    state = fresh()
    torch.cuda.synchronize()
    q = torch.randn(sum(lens), H, D, device="cuda").to(torch.bfloat16)
    kv = torch.randn(sum(lens), K, D, device="cuda").to(torch.bfloat16)
    here = nt.nt_single_attention(p, q, kv, kv, bias=bias)
    torch.cuda.synchronize()
    there = nt.nt_single_attention(p, q, kv, kv, bias=bias, stream=side)
    rotated = nt.nt_qk_norm_rotary(p, q, kv, w, w, table, stream=side.cuda_stream)
    side.synchronize()
    for a, b in zip(here + nt.nt_qk_norm_rotary(p, q, kv, w, w, table), there + rotated):
        np.testing.assert_array_equal(bits(a, torch), bits(b, torch))
    with torch.cuda.stream(side):
        outs = run(state, 1)
    side.synchronize()
    for a, b in zip([bits(x, torch) for x in outs] + [bits(state[0], torch)], want[0]):
        np.testing.assert_array_equal(a, b)


def test_binding_refusals(nt):
    announce("single refusals")
    p = _part(nt, [4, 5])
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    q, k = z(9, 4, 32), z(9, 2, 32)
    with pytest.raises(ValueError):
        nt.nt_single_attention(p, z(8, 4, 32), k, k)
    with pytest.raises(TypeError):
        nt.nt_single_attention(p, q, k.float(), k)
    with pytest.raises(ValueError):
        nt.nt_single_attention(p, q, k, k, bias=z(4, 40))
    with pytest.raises(ValueError):
        nt.nt_single_attention(p, q, k.transpose(1, 2).contiguous().transpose(1, 2), k)
    with pytest.raises(ValueError):
        nt.nt_single_attention(p, q[:1].expand(9, 4, 32), k, k)
    with pytest.raises(nt.NtError):
        nt.nt_single_attention(p, q, z(9, 3, 32), z(9, 3, 32))
    with pytest.raises(nt.NtError):
        nt.nt_single_attention(p, q, k, k, o=q)
    with pytest.raises(nt.NtError):
        nt.nt_single_attention(p, z(9, 4, 136), z(9, 2, 136), z(9, 2, 136))
    with pytest.raises(TypeError):
        nt.nt_single_attention(p, q.half(), k.half(), k.half())
    with pytest.raises(ValueError):
        nt.nt_qk_norm_rotary(p, q, k, w_q=z(32, dt=torch.bfloat16)[:16])
    with pytest.raises(nt.NtError):
        nt.nt_qk_norm_rotary(p, q, k, table=z(9, 64, dt=torch.float32))
    with pytest.raises(nt.NtError):
        nt.nt_qk_norm_rotary(p, q, k, q_out=q.view(-1)[:9 * 128].view(9, 4, 32), k_out=q[:, :2])
    w = torch.zeros(10, device="cuda")
    m, v, _, _ = nt.nt_adamw_states([w])
    with pytest.raises(nt.NtError):
        nt.nt_adamw_step(nt.nt_adamw_tensors([w, w], [w.clone()] * 2, m * 2, v * 2), 1)
    with pytest.raises(nt.NtError):
        nt.nt_adamw_step(nt.nt_adamw_tensors([w], [w.clone()], m, v), 0)
    with pytest.raises(TypeError):
        nt.nt_adamw_tensors([w], [w.bfloat16()], m, v)
    torch.cuda.synchronize()
