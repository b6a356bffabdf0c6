"""GPU parity of the operators between tokens and singles (nt_token_embedding,
nt_residual_norm, nt_token_loss and their gradients) against the float64
oracle, element by element within the bounds that tests/token_bounds.py
derives from the arithmetic."""
import math

import numpy as np
import pytest

import oracle
import token_bounds as tb
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


def _ids(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _within(name, got, ref, bound):
    """Every element within its bound; NaN and infinities in the same places."""
    got = f64(got, torch) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = np.isfinite(ref)
    np.testing.assert_array_equal(got[~fine], ref[~fine], err_msg=name)
    assert np.isfinite(got[fine]).all(), name
    off = np.abs(got - np.where(fine, ref, 0.0))
    over = fine & (off > bound)
    assert not over.any(), (name, int(over.sum()), float((off[fine] / np.broadcast_to(
        np.maximum(bound, 1e-300), off.shape)[fine]).max()))


# ----------------------------------------------------------------- embedding
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,C,scale", [(1, 1, 8, 1.0), (3, 7, 64, 2.0), (65, 33, 72, 0.3),
                                         (130, 1000, 136, 1.0), (17, 300, 384, 19.6),
                                         (9, 40, 1032, -1.5), (5, 12, 4104, 1.0)])
def test_embedding(nt, T, V, C, scale, dtype):
    announce(f"embedding T={T} V={V} C={C} {dtype}")
    rng = np.random.default_rng(T * 1000 + C)
    table, t64 = _dev(rng.normal(size=(V, C)), dtype)
    ids = rng.integers(0, V, size=T)
    ids[rng.random(T) < 0.2] = -1
    if T > 2:
        ids[:3] = [V, -(2 ** 31), 2 ** 31 - 1]
    out = nt.nt_token_embedding(table, _ids(ids), scale=scale)
    ref = oracle.embedding(t64, ids, np.float64(np.float32(scale)))
    _within("out", out, ref, tb.embedding_bound(ref, dtype))


BACK = [(1, 1, 8, 1), (1, 5000, 8, 1), (64, 1, 16, 1), (17, 3, 72, 2), (700, 33, 384, 1),
        (1000, 511, 64, 1), (1000, 513, 128, 1), (2500, 1500, 264, 1), (300, 100000, 40, 1),
        (5000, 7, 520, 3), (40000, 4, 32, 1),
        # either side of the rule for one launch
        (4096, 5, 72, 3), (4097, 5, 72, 3), (40, 4096, 64, 1), (40, 4097, 64, 1), (4096, 2, 8, 2),
        (4100, 2, 8, 2), (4100, 3, 72, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,C,kind", BACK)
def test_embedding_backward(nt, T, V, C, kind, dtype):
    """kind 1: any token; 2: one token in all places; 3: a token in most places.
    The parts of 16 places (more of them from 32,769 places on) end within runs."""
    announce(f"embedding backward T={T} V={V} C={C} kind={kind} {dtype}")
    rng = np.random.default_rng(T + V + C)
    ids = rng.integers(0, V, size=T)
    if kind == 2:
        ids[:] = V - 1
    if kind == 3:
        ids[rng.random(T) < 0.9] = V // 2
    if T > 4 and kind != 2:
        ids[rng.random(T) < 0.1] = -1
        ids[1], ids[2] = V, 2 ** 31 - 1  # tokens of no table row add nothing
    g, g64 = _dev(rng.normal(size=(T, C)), dtype)
    for old in (None, rng.normal(size=(V, C)).astype(np.float32)):
        table = None if old is None else torch.from_numpy(old).cuda()
        got = nt.nt_token_embedding_backward(_ids(ids), g, V, scale=0.5, g_table=table,
                                             accumulate=old is not None)
        old = None if old is None else old.astype(np.float64)
        ref = oracle.embedding_backward(ids, g64, V, 0.5, old)
        _within("g_table", got, ref, tb.embedding_backward_bound(ids, g64, V, 0.5, old) + 1e-30)
        if old is None:  # one order of the sums
            again = nt.nt_token_embedding_backward(_ids(ids), g, V, scale=0.5)
            np.testing.assert_array_equal(bits(got, torch), bits(again, torch))


def test_embedding_backward_nothing(nt):
    """No tokens, and tokens that are all absent: zeros, or what was there."""
    for ids in ([], [-1] * 20, [9] * 20):
        g = torch.full((len(ids), 24), float("nan"), device="cuda")
        out = torch.full((9, 24), 3.0, device="cuda")
        nt.nt_token_embedding_backward(_ids(ids), g, 9, g_table=out, accumulate=True)
        assert bool((out == 3.0).all())
        nt.nt_token_embedding_backward(_ids(ids), g, 9, g_table=out)
        assert bool((out == 0.0).all())


def test_embedding_far_rows(nt):
    """Rows of the table and of the singles past 4 GiB."""
    announce("embedding of 4.6 GB")
    V, C = 140000, 16384
    table = torch.zeros((V, C), dtype=torch.bfloat16, device="cuda")
    table[:, 0] = torch.arange(V, device="cuda") % 251
    table[:, C - 1] = torch.arange(V, device="cuda") // 1000
    ids = torch.arange(V - 1, -1, -1, dtype=torch.int32, device="cuda")
    out = nt.nt_token_embedding(table, ids)
    for row in (0, 1, 70000, V - 1):
        np.testing.assert_array_equal(bits(out[row], torch), bits(table[V - 1 - row], torch))
    assert bool((out[:, 0] == table[:, 0].flip(0)).all())
    assert bool((out[:, C - 1] == table[:, C - 1].flip(0)).all())
    g = nt.nt_token_embedding_backward(ids, out, V)
    assert bool((g[:, 0] == table[:, 0].float()).all())
    assert bool((g[:, C - 1] == table[:, C - 1].float()).all())
    assert bool((g[V - 3:] == table[V - 3:].float()).all())


def test_embedding_rows_behind_stay(nt):
    """Rows behind the last token, and behind the table, are left as they were."""
    big = torch.full((12, 40), 7.0, device="cuda")
    table = torch.ones((5, 40), device="cuda")
    nt.nt_token_embedding(table, _ids([0, 4, -1]), out=big[:3])
    assert bool((big[3:] == 7.0).all()) and bool((big[:2] == 1.0).all())
    nt.nt_token_embedding_backward(_ids([0, 4, -1]), big[:3], 5, g_table=big[4:9])
    assert bool((big[9:] == 7.0).all()) and bool((big[3] == 7.0).all())
    assert bool((big[4] == 1.0).all()) and bool((big[5:8] == 0.0).all())


# ---------------------------------------------------------------------- norm
WIDTHS = [8, 64, 72, 128, 136, 384, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


def _norm_inputs(rng, T, C, dtype, residual):
    x, _ = _dev(rng.normal(size=(T, C)), dtype)
    r = _dev(rng.normal(size=(T, C)) * 2, dtype)[0] if residual else None
    w, w64 = _dev(1.0 + 0.2 * rng.normal(size=C))
    return x, r, w, w64


def _sum_bits(x, r):
    """The stored sum: the fp32 sum of two stored values, rounded once."""
    s = f64(x, torch).astype(np.float32) + f64(r, torch).astype(np.float32)
    return oracle.bf16_bits(s.astype(np.float64)) if x.dtype == torch.bfloat16 else s.view(np.uint32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", WIDTHS)
def test_residual_norm(nt, C, dtype):
    for T in (1, 5, 33) if C <= 2048 else (1, 3):
        announce(f"norm T={T} C={C} {dtype}")
        rng = np.random.default_rng(T * 100 + C)
        for residual in (False, True):
            x, r, w, w64 = _norm_inputs(rng, T, C, dtype, residual)
            for weight, v in ((w, w64), (None, None)):
                y, h = nt.nt_residual_norm(x, weight, residual=r, eps=1e-5)
                if residual:
                    np.testing.assert_array_equal(bits(h, torch), _sum_bits(x, r))
                else:
                    assert h is x
                ref = oracle.residual_norm(f64(h, torch), v, np.float64(np.float32(1e-5)))
                _within("y", y, ref, tb.norm_bound(ref, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,group", [(8, 0), (8, 8), (72, 0), (72, 8), (128, 128), (384, 128),
                                     (384, 0), (1024, 32), (1024, 512), (1536, 512), (4096, 0),
                                     (4096, 128), (8192, 256), (8200, 0), (16384, 0), (16384, 64)])
def test_residual_norm_8bit(nt, C, group, dtype):
    for T in (1, 7, 33) if C <= 2048 else (1, 3):
        announce(f"norm 8 bits T={T} C={C} group={group} {dtype}")
        rng = np.random.default_rng(T * 100 + C + group)
        x, r, w, w64 = _norm_inputs(rng, T, C, dtype, True)
        x[0] *= 1e-30 if dtype == "f32" else 1.0  # small scales beside ordinary ones
        codes, scales, h = nt.nt_residual_norm_8bit(x, w, residual=r, group=group)
        y64 = oracle.residual_norm(f64(h, torch), w64, np.float64(np.float32(1e-6)))
        n = group or C
        pieces = y64.reshape(T, C // n, n)
        top = np.abs(pieces).max(2) / 448.0
        assert tuple(scales.shape) == top.shape
        _within("scales", scales, top, tb.norm_bound(y64, "f32").reshape(pieces.shape).max(2) / 448
                + 4 * tb.U * top)
        s = f64(scales, torch)[:, :, None]
        got = codes.float().cpu().numpy().astype(np.float64).reshape(pieces.shape) * s
        off = np.abs(got - pieces)
        bound = np.maximum(tb.E4M3_HALF * np.abs(pieces), tb.E4M3_LEAST_HALF * s) \
            + (C + 16) * tb.U * np.abs(pieces)
        assert (off <= bound).all(), float((off / bound).max())
        assert (np.abs(codes.float().cpu().numpy()).reshape(pieces.shape).max(2) == 448.0).all()


def test_residual_norm_8bit_small_and_zero(nt):
    """Rows of zeros have scale 0 and codes 0; scales down to fp32's subnormal ones."""
    w = torch.tensor([1e-38, 2e-38, -3e-38, 0.0, 5e-39, 1e-37, 1e-36, 1.5e-38], device="cuda")
    x = torch.ones((2, 8), device="cuda")
    x[1] = 0.0
    codes, scales, _ = nt.nt_residual_norm_8bit(x, w, eps=0.25)
    y = w.double().cpu().numpy() / math.sqrt(1.25)
    got = codes[0].double().cpu().numpy() * float(scales[0, 0].double())
    assert np.abs(got - y).max() <= 2.0 ** -4 * np.abs(y).max()
    assert float(codes[0].float().abs().max()) == 448.0
    assert bool((codes[1].float() == 0).all()) and float(scales[1, 0]) == 0.0


def test_residual_norm_not_finite(nt):
    """A NaN or an infinity stays within its row (and code), and leaves the scale."""
    x = torch.randn((4, 256), device="cuda")
    w = torch.ones(256, device="cuda")
    w[200] = float("inf")
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    y, _ = nt.nt_residual_norm(x, w)
    codes, scales, _ = nt.nt_residual_norm_8bit(x, w, group=128)
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[2, 5]))
    assert bool(torch.isfinite(y[[0, 3]][:, :200]).all()) and bool(torch.isinf(y[0, 200]))
    assert bool(torch.isnan(codes[1].float()).all()) and float(scales[1, 0]) == 0.0
    assert bool(torch.isnan(codes[0, 200].float())) and bool(torch.isfinite(scales).all())
    assert float(codes[0, 128:200].float().abs().max()) <= 448.0 and float(scales[0, 1]) > 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_residual_norm_in_place(nt, dtype):
    rng = np.random.default_rng(5)
    x, r, w, _ = _norm_inputs(rng, 40, 320, dtype, True)
    y, h = nt.nt_residual_norm(x, w, residual=r)
    a, b = x.clone(), r.clone()
    y2, h2 = nt.nt_residual_norm(a, w, residual=b, h=b, y=a)  # the sum in the residual's place
    assert y2 is a and h2 is b
    for p, q in ((y, y2), (h, h2)):
        np.testing.assert_array_equal(bits(p, torch), bits(q, torch))
    a, b = x.clone(), r.clone()
    y3, h3 = nt.nt_residual_norm(a, w, residual=b, h=a, y=b)
    np.testing.assert_array_equal(bits(y, torch), bits(y3, torch))
    np.testing.assert_array_equal(bits(h, torch), bits(h3, torch))
    a = x.clone()
    y4, _ = nt.nt_residual_norm(a, w, y=a)
    np.testing.assert_array_equal(bits(nt.nt_residual_norm(x, w)[0], torch), bits(y4, torch))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", WIDTHS)
def test_residual_norm_backward(nt, C, dtype):
    for T in (1, 6, 131) if C <= 2048 else (1, 3):
        announce(f"norm backward T={T} C={C} {dtype}")
        rng = np.random.default_rng(T * 100 + C)
        h, h64 = _dev(rng.normal(size=(T, C)) * 2, dtype)
        g_y, gy64 = _dev(rng.normal(size=(T, C)), dtype)
        g_h, gh64 = _dev(rng.normal(size=(T, C)), dtype)
        w, w64 = _dev(1.0 + 0.2 * rng.normal(size=C))
        for both in (False, True):
            for weight, v in ((w, w64), (None, None)):
                g, g_w = nt.nt_residual_norm_backward(h, g_y, weight, g_h=g_h if both else None)
                ref, ref_w = oracle.residual_norm_backward(h64, gy64, v, gh64 if both else None,
                                                           np.float64(np.float32(1e-6)))
                b, b_w = tb.norm_backward_bound(h64, gy64, v, gh64 if both else None, ref, dtype)
                _within("g", g, ref, b)
                if weight is None:
                    assert g_w is None
                else:
                    _within("g_w", g_w, ref_w, b_w)
        a = g_y.clone()
        g2, _ = nt.nt_residual_norm_backward(h, a, None, g_h=g_h, g=a)
        np.testing.assert_array_equal(bits(g, torch), bits(g2, torch))
        a = g_h.clone()
        g2, _ = nt.nt_residual_norm_backward(h, g_y, None, g_h=a, g=a)
        np.testing.assert_array_equal(bits(g, torch), bits(g2, torch))


def test_residual_norm_many_rows(nt):
    """More rows than the gradient's workgroups take at a time, and none."""
    rng = np.random.default_rng(9)
    T, C = 5000, 256
    h, h64 = _dev(rng.normal(size=(T, C)), "bf16")
    g_y, gy64 = _dev(rng.normal(size=(T, C)), "bf16")
    w, w64 = _dev(1.0 + 0.2 * rng.normal(size=C))
    g, g_w = nt.nt_residual_norm_backward(h, g_y, w)
    ref, ref_w = oracle.residual_norm_backward(h64, gy64, w64, None, np.float64(np.float32(1e-6)))
    b, b_w = tb.norm_backward_bound(h64, gy64, w64, None, ref, "bf16")
    _within("g", g, ref, b)
    _within("g_w", g_w, ref_w, b_w)
    again = nt.nt_residual_norm_backward(h, g_y, w)[1]
    np.testing.assert_array_equal(bits(g_w, torch), bits(again, torch))
    none = torch.empty((0, 40), device="cuda")
    y, h0 = nt.nt_residual_norm(none, torch.ones(40, device="cuda"), residual=none)
    assert y.shape == (0, 40) and h0.shape == (0, 40)
    g, g_w = nt.nt_residual_norm_backward(none, none, torch.ones(40, device="cuda"))
    assert g.shape == (0, 40) and bool((g_w == 0).all())


def test_residual_norm_far_rows(nt):
    """Rows past 4 GiB: the last ones are as those alone."""
    announce("norm of 4.6 GB")
    T, C, some = 140000, 16384, 5
    rng = np.random.default_rng(4)
    last, _ = _dev(rng.normal(size=(some, C)), "bf16")
    w, _ = _dev(1.0 + 0.2 * rng.normal(size=C))
    x = torch.zeros((T, C), dtype=torch.bfloat16, device="cuda")
    x[T - some:] = last
    y, h = nt.nt_residual_norm(x, w, residual=x)
    y1, h1 = nt.nt_residual_norm(last, w, residual=last)
    codes, scales, _ = nt.nt_residual_norm_8bit(h, w)
    c1, s1, _ = nt.nt_residual_norm_8bit(h1, w)
    g, _ = nt.nt_residual_norm_backward(h, x, w)
    g1, _ = nt.nt_residual_norm_backward(h1, last, w)
    for a, b in ((y, y1), (h, h1), (codes.view(torch.uint8), c1.view(torch.uint8)), (scales, s1),
                 (g, g1)):
        assert bool((a[T - some:] == b).all()) and bool((a[:T - some] == 0).all())


# ---------------------------------------------------------------------- loss
def _loss_inputs(rng, T, V, C, dtype, absent=0.2, spread=2.0):
    x, x64 = _dev(rng.normal(size=(T, C)), dtype)
    W, W64 = _dev(rng.normal(size=(V, C)) * spread / math.sqrt(C), dtype)
    ids = rng.integers(0, V, size=T)
    ids[rng.random(T) < absent] = -1
    ids[T // 2] = V - 1
    return x, x64, W, W64, ids


LOSS = [(1, 1, 8), (1, 2, 64), (2, 127, 72), (5, 128, 136), (32, 129, 40), (17, 70001, 24), (16, 65, 264), (31, 1000, 384),
        (33, 33, 8), (64, 257, 64), (130, 300, 200), (257, 128, 1032), (300, 1301, 128)]


def _check_loss(nt, x, x64, W, W64, ids, scale, dtype):
    nll, lse = nt.nt_token_loss(x, W, _ids(ids), scale=scale)
    rn, rl = oracle.token_loss(x64, W64, ids, np.float64(np.float32(scale)))
    bn, bl = tb.loss_bound(x64, W64, ids, rl, scale)
    _within("lse", lse, rl, bl)
    _within("nll", nll, rn, bn)
    return lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,C", LOSS)
def test_token_loss(nt, T, V, C, dtype):
    announce(f"loss T={T} V={V} C={C} {dtype}")
    rng = np.random.default_rng(T + V + C)
    x, x64, W, W64, ids = _loss_inputs(rng, T, V, C, dtype)
    for scale in (1.0, -0.3):
        _check_loss(nt, x, x64, W, W64, ids, scale, dtype)


def test_token_loss_many_tiles(nt):
    """Enough tiles for the widest ones, with partial ones at both ends."""
    announce("loss T=3900 V=4300")
    rng = np.random.default_rng(1)
    x, x64, W, W64, ids = _loss_inputs(rng, 3900, 4300, 72, "bf16", absent=0.01)
    _check_loss(nt, x, x64, W, W64, ids, 1.0, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,C", [(3, 130, 4104), (16, 1000, 2056), (31, 200, 2056), (20, 66000, 520)])
def test_token_loss_few_tokens(nt, T, V, C, dtype):
    """Rows of x that LDS holds in stretches only, and more rows of W than the launched
    waves take at a time."""
    announce(f"loss T={T} V={V} C={C} {dtype}")
    rng = np.random.default_rng(T + V + C)
    x, x64, W, W64, ids = _loss_inputs(rng, T, V, C, dtype)
    _check_loss(nt, x, x64, W, W64, ids, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_token_loss_passes(nt, dtype):
    """More tokens than a pass takes, forward and back; the last pass has no target at
    all in its first half."""
    announce(f"loss T=140000 {dtype}")
    rng = np.random.default_rng(8)
    x, x64, W, W64, ids = _loss_inputs(rng, 140000, 24, 16, dtype, absent=0.5)
    ids[131072:135000] = -1
    lse = _check_loss(nt, x, x64, W, W64, ids, 1.0, dtype)
    _check_backward(nt, x, x64, W, W64, ids, lse, dtype, 1.0, rng, True, True)


@pytest.mark.parametrize("T,V,C,absent,what", [
    (6140, 6130, 8, 0.01, "the logits"),
    (36860, 16, 1024, 0.97, "g_x"),
    (40, 36860, 1024, 0.0, "g_W")])
def test_token_loss_wide_tiles_f32(nt, T, V, C, absent, what):
    announce(f"loss T={T} V={V} C={C} f32: wide tiles of {what}")
    rng = np.random.default_rng(12)
    x, x64, W, W64, ids = _loss_inputs(rng, T, V, C, "f32", absent=absent)
    lse = _check_loss(nt, x, x64, W, W64, ids, 1.0, "f32")
    _check_backward(nt, x, x64, W, W64, ids, lse, "f32", 1.0, rng, False, False)


@pytest.mark.parametrize("T", [5, 40])
def test_token_loss_far_rows(nt, T):
    """Rows of W past 4 GiB: all are zeros but the last ones, so that the logits of the
    others are 0 and the gradient of the others is p0 x, p0 = exp(-lse)."""
    V, C, some = 140000, 16384, 300
    announce(f"loss T={T} V={V} C={C}")
    rng = np.random.default_rng(T)
    x, x64 = _dev(rng.normal(size=(T, C)), "bf16")
    last, last64 = _dev(rng.normal(size=(some, C)) * 4 / math.sqrt(C), "bf16")
    W = torch.zeros((V, C), dtype=torch.bfloat16, device="cuda")
    W[V - some:] = last
    ids = rng.integers(V - some, V, size=T)
    ids[1] = -1
    ids[2] = 7
    nll, lse = nt.nt_token_loss(x, W, _ids(ids))
    # the last rows and a zero one, which counts for all the others
    few = np.concatenate([np.zeros((1, C)), last64])
    z = x64 @ few.T
    top = z.max(1, keepdims=True)
    count = np.r_[V - some, np.ones(some)]
    want = (top[:, 0] + np.log((np.exp(z - top) * count).sum(1))) * (ids >= 0)
    at = np.where(ids >= V - some, ids - (V - some) + 1, 0)
    err = tb._logit_error(x64, few, 1.0, want)
    p = np.exp(z - want[:, None]) * count
    # as in token_bounds.loss_bound, with a weight for each row
    bl = ((p * err).sum(1) + (V + 8) * tb.U + 8 * tb.U * (1 + np.abs(want))) * (ids >= 0)
    _within("lse", lse, want, bl)
    _within("nll", nll, np.where(ids >= 0, want - z[np.arange(T), at], 0.0),
            bl + err[np.arange(T), at] * (ids >= 0))
    if T > 5:
        return
    g = torch.ones(T, device="cuda")
    g_x, g_W = nt.nt_token_loss_backward(x, W, _ids(ids), lse, g)
    l64 = f64(lse, torch)
    local = np.where(ids < 0, -1, at)
    # one zero row as the vocabulary has it: its gradient is that of every zero row but
    # the seventh, which is a target
    rx, rW = oracle.token_loss_backward(x64, few, local, l64, np.ones(T))
    bx, bW = tb.loss_backward_bound(x64, few, local, l64, np.ones(T), None, 1.0, None, rx, "bf16")
    # the zero rows add nothing to g_x, the longer sum of the product nothing but zeros
    _within("g_x", g_x, rx, bx)
    _within("g_W", g_W[V - some:], rW[1:], bW[1:])
    _within("g_W[7]", g_W[7:8], rW[:1], bW[:1])
    rest = np.exp(-l64) * (ids >= 0) @ x64
    _within("g_W[V - some - 1]", g_W[V - some - 1:V - some], rest[None], bW[:1])


@pytest.mark.parametrize("T", [20, 200])
def test_token_loss_absent_rows(nt, T):
    """Rows without a target reach nothing, whatever they hold; all of them, too."""
    rng = np.random.default_rng(T)
    x, x64, W, W64, ids = _loss_inputs(rng, T, 77, 64, "bf16", absent=0.7)
    clean = nt.nt_token_loss(x, W, _ids(ids))
    g = torch.rand(T, device="cuda")
    want = nt.nt_token_loss_backward(x, W, _ids(ids), clean[1], g, g_lse=g)
    gone = torch.from_numpy(ids < 0).cuda()
    x[gone] = float("nan")
    lse, g2 = clean[1].clone(), g.clone()
    lse[gone] = float("nan")
    g2[gone] = float("inf")
    got = nt.nt_token_loss(x, W, _ids(ids))
    grads = nt.nt_token_loss_backward(x, W, _ids(ids), lse, g2, g_lse=g2)
    for a, b in zip((*clean, *want), (*got, *grads)):
        np.testing.assert_array_equal(bits(a, torch), bits(b, torch))
    assert bool((got[0][gone] == 0).all()) and bool((grads[0][gone] == 0).all())
    none = _ids([-1] * T)
    nll, lse = nt.nt_token_loss(x, W, none)
    g_x, g_W = nt.nt_token_loss_backward(x, W, none, lse, g)
    assert all(bool((t == 0).all()) for t in (nll, lse, g_x, g_W))


def test_token_loss_foreign_targets(nt):
    """A target that the vocabulary does not hold: nll NaN, the others as they were;
    its gradients are NaN, the other tokens' g_x is not touched."""
    rng = np.random.default_rng(3)
    x, x64, W, W64, ids = _loss_inputs(rng, 40, 50, 64, "f32", absent=0.0)
    a = nt.nt_token_loss(x, W, _ids(ids))
    g = torch.ones(40, device="cuda")
    gx = nt.nt_token_loss_backward(x, W, _ids(ids), a[1], g)[0]
    ids2 = ids.copy()
    ids2[7] = 50
    b = nt.nt_token_loss(x, W, _ids(ids2))
    gx2, gW2 = nt.nt_token_loss_backward(x, W, _ids(ids2), b[1], g)
    others = [i for i in range(40) if i != 7]
    assert math.isnan(float(b[0][7])) and bool((b[1] == a[1]).all())
    assert bool((b[0][others] == a[0][others]).all()) and bool((gx2[others] == gx[others]).all())
    assert bool(torch.isnan(gx2[7]).all()) and bool(torch.isnan(gW2).all())


def test_token_loss_large_logits(nt):
    """Logits of thousands, equal ones, and one that leaves the others nothing."""
    x = torch.zeros((3, 16), device="cuda")
    x[0, 0], x[1, 1] = 1000.0, 3e4
    W = torch.zeros((300, 16), device="cuda")
    W[:, 0] = 5.0
    W[123, 1] = 1.0
    nll, lse = nt.nt_token_loss(x, W, _ids([7, 123, 299]))
    ref = [5000.0 + math.log(300), 3e4, math.log(300)]
    np.testing.assert_allclose(lse.cpu().numpy(), ref, rtol=2.0 ** -21)
    np.testing.assert_allclose(nll.cpu().numpy(), [math.log(300), 0.0, math.log(300)],
                               rtol=0, atol=5000 * 2.0 ** -21)
    # Only that logit counts: its power's exponent r is what rounding the base of 43,281 lost,
    # at most 2^-9; nll = (log2(2^r) - r) ln 2. The power is off by one step at most (2^-23
    # of its value, so 1.45 times 2^-23 in its logarithm), the logarithm near 0 by less.
    assert abs(float(nll[1])) <= 2.0 ** -21


def test_token_loss_infinite_logits(nt):
    """Rows of W that give -inf have no weight; where all do, nothing is left."""
    x = torch.ones((34, 8), device="cuda")
    W = torch.randn((200, 8), device="cuda")
    W[50:60, 2] = -math.inf
    ids = np.full(34, 3)
    keep = torch.cat([W[:50], W[60:]])
    a, b = nt.nt_token_loss(x, W, _ids(ids)), nt.nt_token_loss(x, keep, _ids(ids))
    np.testing.assert_allclose(a[1].cpu(), b[1].cpu(), rtol=0, atol=200 * tb.U * 8)
    W[:, 2] = -math.inf
    assert bool((nt.nt_token_loss(x, W, _ids(ids))[1] == -math.inf).all())


BACKWARD = [(1, 1, 8), (1, 300, 64), (2, 127, 72), (33, 33, 8), (64, 257, 64), (130, 300, 200),
            (257, 128, 1032), (300, 1301, 128), (700, 40, 256), (90, 3000, 64)]


def _check_backward(nt, x, x64, W, W64, ids, lse, dtype, scale, rng, both, accumulate):
    T, V = len(ids), len(W)
    g_nll, gn64 = _dev(rng.normal(size=T) / T)
    g_lse, gl64 = _dev(rng.normal(size=T) / T) if both else (None, None)
    old, old64 = _dev(rng.normal(size=W.shape) * 1e-2) if accumulate else (None, None)
    g_x, g_W = nt.nt_token_loss_backward(x, W, _ids(ids), lse, g_nll, g_lse=g_lse, scale=scale,
                                         g_W=old, accumulate=accumulate)
    s = np.float64(np.float32(scale))
    rx, rW = oracle.token_loss_backward(x64, W64, ids, f64(lse, torch), gn64, gl64, s, old64)
    bx, bW = tb.loss_backward_bound(x64, W64, ids, f64(lse, torch), gn64, gl64, s, old64, rx, dtype)
    _within("g_x", g_x, rx, bx)
    _within("g_W", g_W, rW, bW)
    return g_nll, g_lse, g_x, g_W


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,C", BACKWARD)
def test_token_loss_backward(nt, T, V, C, dtype):
    announce(f"loss backward T={T} V={V} C={C} {dtype}")
    rng = np.random.default_rng(T + V + C)
    x, x64, W, W64, ids = _loss_inputs(rng, T, V, C, dtype)
    for scale, both, accumulate in ((1.0, False, False), (-0.3, True, True)):
        lse = nt.nt_token_loss(x, W, _ids(ids), scale=scale)[1]
        g_nll, g_lse, g_x, g_W = _check_backward(nt, x, x64, W, W64, ids, lse, dtype, scale, rng,
                                                 both, accumulate)
        gx2, gW2 = nt.nt_token_loss_backward(x, W, _ids(ids), lse, g_nll, g_lse=g_lse, scale=scale,
                                             weight_grad=False)
        assert gW2 is None
        np.testing.assert_array_equal(bits(g_x, torch), bits(gx2, torch))


@pytest.mark.parametrize("T,V,C,absent,what", [
    (3900, 4300, 64, 0.01, "wide tiles of the logits"),
    (7100, 40, 2056, 0.9, "wide tiles of g_x"),
    (60, 8100, 2056, 0.0, "wide tiles of g_W"),
    (131000, 1100, 64, 0.998, "pieces of the vocabulary")])
def test_token_loss_backward_large(nt, T, V, C, absent, what):
    announce(f"loss backward T={T} V={V} C={C}: {what}")
    rng = np.random.default_rng(T)
    x, x64, W, W64, ids = _loss_inputs(rng, T, V, C, "bf16", absent=absent)
    lse = nt.nt_token_loss(x, W, _ids(ids))[1]
    _check_backward(nt, x, x64, W, W64, ids, lse, "bf16", 1.0, rng, False, False)


def test_token_loss_gradient_against_differences(nt):
    """The fp32 gradients against central differences of the loss itself."""
    rng = np.random.default_rng(11)
    x, x64, W, W64, ids = _loss_inputs(rng, 20, 45, 16, "f32")
    lse = nt.nt_token_loss(x, W, _ids(ids))[1]
    g_nll, gn64 = _dev(rng.normal(size=20))
    g_x, g_W = nt.nt_token_loss_backward(x, W, _ids(ids), lse, g_nll)
    step = 1e-5

    def loss(a, b):
        return float(oracle.token_loss(a, b, ids)[0] @ gn64)

    for of, grad in ((x64, g_x), (W64, g_W)):
        for _ in range(12):
            i = tuple(rng.integers(0, n) for n in of.shape)
            keep = of[i]
            of[i] = keep + step
            up = loss(x64, W64)
            of[i] = keep - step
            down = loss(x64, W64)
            of[i] = keep
            # the difference's error: step^2 times the third derivative, and fp32's
            assert abs(float(grad[i]) - (up - down) / (2 * step)) < 1e-4


def test_token_loss_nothing(nt):
    W = torch.randn((30, 16), device="cuda")
    x, ids, none = torch.empty((0, 16), device="cuda"), _ids([]), torch.empty(0, device="cuda")
    nll, lse = nt.nt_token_loss(x, W, ids)
    assert nll.shape == (0,) and lse.shape == (0,)
    old = torch.full((30, 16), 2.0, device="cuda")
    g_x, g_W = nt.nt_token_loss_backward(x, W, ids, lse, none, g_W=old, accumulate=True)
    assert g_x.shape == (0, 16) and bool((g_W == 2.0).all())
    assert bool((nt.nt_token_loss_backward(x, W, ids, lse, none, g_W=old)[1] == 0.0).all())


# ----------------------------------------------------------------- as a whole
def _step(nt, table, tokens, targets, w, out):
    """Tokens to singles, a residual norm, the loss, and back: the table's
    gradient is that of both of its uses."""
    n = tokens.shape[0]
    s0 = nt.nt_token_embedding(table, tokens, scale=2.0)
    y, h = nt.nt_residual_norm(s0, w, residual=s0)
    nll, lse = nt.nt_token_loss(y, table, targets)
    g = torch.full_like(nll, 1.0 / n)
    g_y, g_table = nt.nt_token_loss_backward(y, table, targets, lse, g, g_W=out)
    g_h, g_w = nt.nt_residual_norm_backward(h, g_y, w)
    g_s0 = g_h + g_h
    nt.nt_token_embedding_backward(tokens, g_s0, table.shape[0], scale=2.0, g_table=g_table,
                                   accumulate=True)
    return nll, g_table, g_w


def test_together(nt):
    """A tied table through all of them in fp32, against float64 autograd, and the
    optimizer's step on its gradient."""
    torch.manual_seed(0)
    V, C, T = 61, 64, 150
    table = torch.randn((V, C), device="cuda") * 0.3
    w = 1.0 + 0.1 * torch.randn(C, device="cuda")
    ids = torch.randint(0, V, (T + 1,), device="cuda", dtype=torch.int32)
    ids[70] = -1  # an absent token, which is nobody's target
    tokens, targets = ids[:-1], ids[1:]  # the next token, at an address between words of 16 bytes
    nll, g_table, g_w = _step(nt, table, tokens, targets, w, torch.empty_like(table))

    t64, w64 = table.double().cpu().requires_grad_(), w.double().cpu().requires_grad_()
    i, t = ids[:-1].long().cpu(), ids[1:].long().cpu()
    s0 = 2.0 * t64[i.clamp(min=0)] * (i >= 0)[:, None]
    h = 2 * s0
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * w64
    lp = torch.log_softmax(y @ t64.t(), 1)
    ref = -lp.gather(1, t.clamp(min=0)[:, None])[:, 0] * (t >= 0)
    (ref.sum() / T).backward()
    # fp32 sums of at most 150 terms of a few units: 2^-24 times some hundreds
    assert float((nll.double().cpu() - ref.detach()).abs().max()) < 2e-4
    for got, want in ((g_table, t64.grad), (g_w, w64.grad)):
        assert float((got.double().cpu() - want).abs().max()) < 1e-4 * float(want.abs().max()) + 1e-6

    m, v, _, _ = nt.nt_adamw_states([table, w])
    before = table.clone()
    tensors = nt.nt_adamw_tensors([table, w], [g_table, g_w], m, v)
    nt.nt_adamw_step(tensors, 1, lr=1e-2)
    assert bool((table != before).any())
    after = nt.nt_token_loss(nt.nt_residual_norm(nt.nt_token_embedding(table, tokens), w)[0], table,
                             targets)[0]
    assert bool(torch.isfinite(after).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(nt, dtype):
    """All operators in one graph, replayed on new inputs with eager calls between:
    every replay as the eager calls."""
    dt = getattr(torch, DT[dtype])
    V, C, T = 600, 136, 90
    torch.manual_seed(1)
    table = (torch.randn((V, C), device="cuda") * 0.3).to(dt)
    w = torch.ones(C, device="cuda")
    ids = torch.randint(-1, V, (T + 4,), device="cuda", dtype=torch.int32)
    out = torch.empty((V, C), device="cuda")
    tokens, targets = ids[:T], ids[4:]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(2):
            _step(nt, table, tokens, targets, w, out)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(nt, table, tokens, targets, w, out)
    for k in range(4):
        ids.copy_(torch.randint(-1 - 300 * (k % 2), V, (T + 4,), device="cuda", dtype=torch.int32))
        table.copy_((torch.randn((V, C), device="cuda") * 0.3).to(dt))
        graph.replay()
        torch.cuda.synchronize()
        held = [t.clone() for t in got]
        want = _step(nt, table, tokens, targets, w, torch.empty_like(out))
        for a, b in zip(held, want):
            np.testing.assert_array_equal(bits(a, torch), bits(b, torch))


def test_other_streams_at_once(nt):
    """Two streams with workspaces of their own give what one gives."""
    torch.manual_seed(2)
    V, C, T = 900, 128, 400
    table = (torch.randn((V, C), device="cuda") * 0.3).to(torch.bfloat16)
    w = torch.ones(C, device="cuda")
    batches = [torch.randint(-1, V, (T + 4,), device="cuda", dtype=torch.int32) for _ in range(2)]
    want = [_step(nt, table, b[:T], b[4:], w, torch.empty((V, C), device="cuda")) for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    got = []
    for b, s in zip(batches, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([_step(nt, table, b[:T], b[4:], w, torch.empty((V, C), device="cuda"))
                        for _ in range(5)][-1])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for p, q in zip(a, b):
            np.testing.assert_array_equal(bits(p, torch), bits(q, torch))
    # a stream by its handle, and a given workspace
    need = nt.nt_token_loss_workspace_bytes(T, V, C, "bf16")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    x = nt.nt_token_embedding(table, batches[0][:T], stream=streams[0])
    torch.cuda.synchronize()
    a = nt.nt_token_loss(x, table, batches[0][4:], workspace=ws, stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    b = nt.nt_token_loss(x, table, batches[0][4:])
    np.testing.assert_array_equal(bits(a[0], torch), bits(b[0], torch))


def test_binding_refusals(nt):
    x = torch.randn((6, 16), device="cuda")
    W = torch.randn((9, 16), device="cuda")
    ids = _ids([0, 1, 2, 3, 4, 5])
    g = torch.ones(6, device="cuda")
    lse = torch.ones(6, device="cuda")
    bad = [
        lambda: nt.nt_token_embedding(W, ids.long()),
        lambda: nt.nt_token_embedding(W.t(), ids),
        lambda: nt.nt_token_embedding(W, ids, out=torch.empty((6, 8), device="cuda")),
        lambda: nt.nt_token_embedding(W.half(), ids),
        lambda: nt.nt_token_embedding(W.cpu(), ids),
        lambda: nt.nt_token_embedding(W, ids.cpu()),
        lambda: nt.nt_token_embedding(W, ids, out=W[:6]),
        lambda: nt.nt_token_embedding_backward(ids[:5], x, 9),
        lambda: nt.nt_token_embedding_backward(ids, x, 9, accumulate=True),
        lambda: nt.nt_token_embedding_backward(ids, x, 9, g_table=W[:8]),
        lambda: nt.nt_residual_norm(x[:, :8]),
        lambda: nt.nt_residual_norm(x, g),
        lambda: nt.nt_residual_norm(x, residual=x.bfloat16()),
        lambda: nt.nt_residual_norm(x, h=torch.empty_like(x)),
        lambda: nt.nt_residual_norm_8bit(x, group=3),
        lambda: nt.nt_residual_norm_8bit(x, group=-8),
        lambda: nt.nt_residual_norm_8bit(x, scales=torch.empty(6, device="cuda")),
        lambda: nt.nt_residual_norm_backward(x, x[:5]),
        lambda: nt.nt_residual_norm_backward(x, x, g=x),
        lambda: nt.nt_token_loss(x, W[:, :8].contiguous(), ids),
        lambda: nt.nt_token_loss(x, W.bfloat16(), ids),
        lambda: nt.nt_token_loss(x, W, ids[:3]),
        lambda: nt.nt_token_loss(x, W, ids, workspace=torch.empty(4, device="cuda")),
        lambda: nt.nt_token_loss(x, W, ids, nll=g, lse=g),
        lambda: nt.nt_token_loss(x, W, ids, scale=float("nan")),
        lambda: nt.nt_token_loss_backward(x, W, ids, lse, None),
        lambda: nt.nt_token_loss_backward(x, W, ids, lse, g, accumulate=True),
        lambda: nt.nt_token_loss_backward(x, W, ids, lse, g, g_W=W),
        lambda: nt.nt_token_loss_backward(x, W, ids, lse, g, g_W=W.clone(), weight_grad=False),
    ]
    keep = W.clone()
    for k, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, nt.NtError)):
            call()
            raise AssertionError(f"call {k} was not refused")
    assert bool((W == keep).all())
