"""GPU tests of calls at the edge of what the single operators take: scales that are
negative or zero, token distances and arrays past 32 bits, the most heads, samples
without rows or columns, a bias without its gradient."""
import math

import numpy as np
import pytest

import oracle
import single_bounds as sb
from gpu_util import announce, bits, f64
from test_gpu_single import DT, _attention_inputs, _dev, _part, _within, nt  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SCALED = [
    ([70, 33], None, 2, 2, 32, "none", True, "bf16", "split"),
    ([70, 33], None, 4, 2, 40, "plain", False, "f32", "split"),
    ([70, 33], None, 4, 2, 64, "masked", True, "bf16", "split"),
    ([1, 1, 2], [3000, 900, 513], 4, 2, 64, "none", False, "f32", "split"),  # parts of keys
    ([1, 1, 2], [3000, 900, 513], 4, 2, 64, "plain", False, "bf16", "split"),
]


@pytest.mark.parametrize("scale", [-0.3, 0.0])
@pytest.mark.parametrize("case", SCALED)
def test_scales(nt, case, scale):  # noqa: F811
    """A negative scale is the positive one with -q; zero leaves the bias alone."""
    rows, cols, H, K, D, kind, causal, dtype, layout = case
    announce(f"attention scale {scale} {case}")
    rng = np.random.default_rng(91)
    c, (q, k, v, b), (q64, k64, v64, b64), _ = _attention_inputs(rng, case)
    g, g64 = _dev(rng.normal(size=tuple(q.shape)), dtype)
    p = _part(nt, rows, cols)
    o, lse = nt.nt_single_attention(p, q, k, v, bias=b, causal=causal, scale=scale)
    got = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=b, causal=causal, scale=scale)
    torch.cuda.synchronize()
    turn, size = (-1.0, -scale) if scale < 0 else (1.0, scale)
    ro, rl = oracle.attention(rows, c, turn * q64, k64, v64, b64, causal, size)
    bo, bl = sb.attention_bound(rows, c, turn * q64, k64, v64, ro, rl, b64, causal, size, dtype)
    o64, l64 = f64(o, torch), f64(lse, torch)
    _within("o", o64, ro, bo)
    _within("lse", l64, rl, bl)
    ref = oracle.attention_backward(rows, c, turn * q64, k64, v64, o64, l64, g64, b64, causal, size)
    bound = sb.attention_backward_bound(rows, c, turn * q64, k64, v64, o64, l64, g64, ref[:3], b64,
                                        causal, size, dtype)
    for name, x, r, e in zip(("g_q", "g_k", "g_v", "g_bias"), got, ref, bound):
        if r is not None:
            _within(name, f64(x, torch), turn * r if name == "g_q" else r, e)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_widest_token_distance(nt, dtype):  # noqa: F811
    """q, k and v 2^22 elements from token to token: a tile of 64 (or 128) rows spans
    up to 2 GiB. The results are those of packed arrays."""
    announce(f"attention, widest distance {dtype}")
    t = getattr(torch, DT[dtype])
    n, H, D, ld = 130, 2, 32, 1 << 22
    gen = torch.Generator(device="cuda").manual_seed(92)
    wide = torch.empty(n * ld, dtype=t, device="cuda")
    parts = [torch.as_strided(wide, (n, H, D), (ld, D, 1), H * D * i) for i in range(3)]
    packed = []
    for x in parts:
        y = torch.randn((n, H, D), generator=gen, device="cuda").to(t)
        x.copy_(y)
        packed.append(y)
    g = torch.randn((n, H, D), generator=gen, device="cuda").to(t)
    p = _part(nt, [n])
    outs = []
    for q, k, v in (parts, packed):
        o, lse = nt.nt_single_attention(p, q, k, v, causal=True)
        outs.append((o, lse) + nt.nt_single_attention_backward(p, q, k, v, o, lse, g,
                                                               causal=True)[:3])
    torch.cuda.synchronize()
    for x, y in zip(*outs):
        np.testing.assert_array_equal(bits(x, torch), bits(y, torch))


def test_keys_past_32_bits(nt):  # noqa: F811
    """One new token over 2.2 million kept keys of 1,024 elements: k and v pass 4 GiB
    each. The reference is in 64 bits on the device, piece by piece."""
    announce("attention, keys past 32 bits")
    H, D, cols = 8, 128, [33, 2_200_000]
    Tc = sum(cols)
    gen = torch.Generator(device="cuda").manual_seed(93)
    k, v = (torch.empty((Tc, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (k, v):
        for i in range(0, Tc, 1 << 18):
            x[i:i + (1 << 18)].normal_(generator=gen)
    q = torch.randn((2, H, D), generator=gen, device="cuda").to(torch.bfloat16)
    o, lse = nt.nt_single_attention(_part(nt, [1, 1], cols), q, k, v)
    torch.cuda.synchronize()
    scale, at = 1 / math.sqrt(D), 0
    for i, m in enumerate(cols):
        s = torch.empty((H, m), dtype=torch.float64, device="cuda")
        for j in range(0, m, 1 << 17):
            part = k[at + j:at + min(m, j + (1 << 17))].double()
            s[:, j:j + len(part)] = (part * q[i].double()).sum(-1).t() * scale
        z = torch.logsumexp(s, 1)
        w = torch.exp(s - z[:, None])
        ref = torch.zeros((H, D), dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(ref)
        for j in range(0, m, 1 << 17):
            part = v[at + j:at + min(m, j + (1 << 17))].double()
            wj = w[:, j:j + len(part)].t()[:, :, None]
            ref += (wj * part).sum(0)
            mag += (wj * part.abs()).sum(0)
        # P is rounded to bf16 before its product and o once. Sums: a lane adds 16 powers of a
        # tile at a time over at most 2^21 / (64 parts x 4 lanes) keys, then the parts
        steps = m / 256 + 512
        err = (D + 8 + steps) * sb.U * (1 + float(s.abs().max()))
        e = sb.HALF["bf16"]
        assert bool(((o[i].double() - ref).abs() <= (2 * err + e) * mag + e * ref.abs() + 1e-30).all())
        assert bool(((lse[i].double() - z).abs() <= err + 8 * sb.U * z.abs()).all())
        at += m
        del s, w


def test_the_most_heads(nt):  # noqa: F811
    announce("attention, 4096 heads")
    rng = np.random.default_rng(94)
    for K in (4096, 1):
        case = ([2, 0, 3], None, 4096, K, 8, "plain", True, "bf16", "split")
        rows, _, H, _, D, _, causal, dtype, _ = case
        c, (q, k, v, b), (q64, k64, v64, b64), scale = _attention_inputs(rng, case)
        g, g64 = _dev(rng.normal(size=tuple(q.shape)), dtype)
        p = _part(nt, rows)
        o, lse = nt.nt_single_attention(p, q, k, v, bias=b, causal=causal)
        got = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=b, causal=causal)
        torch.cuda.synchronize()
        ro, rl = oracle.attention(rows, c, q64, k64, v64, b64, causal, scale)
        bo, _ = sb.attention_bound(rows, c, q64, k64, v64, ro, rl, b64, causal, scale, dtype)
        o64, l64 = f64(o, torch), f64(lse, torch)
        _within("o", o64, ro, bo)
        ref = oracle.attention_backward(rows, c, q64, k64, v64, o64, l64, g64, b64, causal, scale)
        bound = sb.attention_backward_bound(rows, c, q64, k64, v64, o64, l64, g64, ref[:3], b64,
                                            causal, scale, dtype)
        for name, x, r, e in zip(("g_q", "g_k", "g_v", "g_bias"), got, ref, bound):
            _within(name, f64(x, torch), r, e)


@pytest.mark.parametrize("rows,cols", [([], []), ([0, 0], [0, 0]), ([0, 3], [0, 0]), ([0, 0], [4, 70])])
def test_nothing_to_attend(nt, rows, cols):  # noqa: F811
    """No samples, no rows, or no columns: o = 0, lse = -inf, gradients of zero."""
    announce(f"attention of nothing {rows} {cols}")
    p = nt.nt_make_partition_rect(rows, cols)
    T, Tc, H, K, D = sum(rows), sum(cols), 4, 2, 32
    make = lambda n, h: torch.randn((n, h, D), device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, g = make(T, H), make(Tc, K), make(Tc, K), make(T, H)
    b = torch.zeros((H, 0), dtype=torch.bfloat16, device="cuda")
    for bias in (None, b):
        o, lse = nt.nt_single_attention(p, q, k, v, bias=bias)
        got = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=bias)
        torch.cuda.synchronize()
        assert bool((o == 0).all()) and bool((lse == -math.inf).all())
        assert all(x is None or bool((x == 0).all()) for x in got)
        table = nt.nt_rotary_table(80, D)
        out = nt.nt_qk_norm_rotary(p, q, k, table=table)
        assert out[0].shape == q.shape and out[1].shape == k.shape
        w = torch.ones(D, device="cuda")
        back = nt.nt_qk_norm_rotary_backward(p, q, k, g, make(Tc, K) * 0, w, w, table)
        torch.cuda.synchronize()
        assert bool((back[3] == 0).all()) and (T > 0 or bool((back[2] == 0).all()))


def test_bias_without_its_gradient(nt):  # noqa: F811
    """The other gradients are those of a call that writes it too."""
    announce("attention, bias without gradient")
    case = ([70, 0, 129], None, 2, 2, 64, "masked", True, "bf16", "split")
    rng = np.random.default_rng(95)
    _, (q, k, v, b), _, _ = _attention_inputs(rng, case)
    g, _ = _dev(rng.normal(size=tuple(q.shape)), "bf16")
    p = _part(nt, case[0])
    o, lse = nt.nt_single_attention(p, q, k, v, bias=b, causal=True)
    with_it = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=b, causal=True)
    without = nt.nt_single_attention_backward(p, q, k, v, o, lse, g, bias=b, causal=True,
                                              bias_grad=False)
    torch.cuda.synchronize()
    assert without[3] is None
    for x, y in zip(with_it[:3], without[:3]):
        np.testing.assert_array_equal(bits(x, torch), bits(y, torch))
