"""Cases of the single attention operators and of the optimizer step.

The operators: norms of queries and keys with the position rotation in the
same pass (forward, backward), attention among the packed singles of each
sample (forward, backward), and AdamW over many tensors. `run` computes them
in plain torch, padded to the longest sample, or, where `own` is true, through
the library.

A case names its lengths as text ("7,12,5"); "cols" is there for rectangular
partitions (queries of the rows attend to the columns). "layout" is "split"
for separate arrays and "fused" where q, k (and v) are parts of one projected
array, as a fused projection leaves them.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0       # largest finite e4m3 value
E4M3_LEAST = 2.0 ** -9  # smallest positive one
STATE_BLOCK = 256      # elements that share a scale


# --------------------------------------------------------------------- cases
def listed():
    return [
        # The smallest training batch: eight short samples, c_s 128 as four heads of 32.
        {"name": "norm one_block", "op": "norm", "lens": "94,97,113,125,66,73,117,125", "heads": 4,
         "kv_heads": 4, "dim": 32, "rot": 32, "interleaved": False, "scaling": "none",
         "layout": "split", "dtype": "bf16", "offset": False},
        # A long packed batch behind a fused projection: shared key heads, half of the
        # head rotated, frequencies scaled by parts for four times the trained length.
        {"name": "norm long fused", "op": "norm", "lens": "8192,4096,2048,1024,512,333,100,79",
         "heads": 32, "kv_heads": 8, "dim": 128, "rot": 64, "interleaved": True,
         "scaling": "parts", "layout": "fused", "dtype": "bf16", "offset": False},
        # The high-variation batch trained in fp32, c_s 384 as twelve heads of 32.
        {"name": "norm_bwd high_variation", "op": "norm_bwd",
         "lens": "22,36,257,120,22,72,84,28,204,24,62,96,71,122,206,440", "heads": 12,
         "kv_heads": 12, "dim": 32, "rot": 32, "interleaved": False, "scaling": "none",
         "layout": "split", "dtype": "f32", "offset": False},
        # The backward of a long batch with wide heads and shared key heads.
        {"name": "norm_bwd long", "op": "norm_bwd", "lens": "8192,4096,2048,1024,512,333,100,79",
         "heads": 16, "kv_heads": 4, "dim": 128, "rot": 128, "interleaved": False,
         "scaling": "linear", "layout": "split", "dtype": "bf16", "offset": False},
        # The tiny fp32 batch: the latency of one call.
        {"name": "attn tiny_fp32", "op": "attn", "lens": "7,12,5,16", "cols": "", "heads": 2,
         "kv_heads": 2, "dim": 8, "bias": "plain", "causal": False, "layout": "split",
         "dtype": "f32"},
        # The near-uniform batch with a bias from the pair state.
        {"name": "attn near_uniform", "op": "attn",
         "lens": "252,237,232,238,241,251,242,232,239,246,251,249,256,235,253,231", "cols": "",
         "heads": 12, "kv_heads": 12, "dim": 32, "bias": "plain", "causal": False,
         "layout": "split", "dtype": "bf16"},
        # One new token of each of sixteen samples over its kept keys and values.
        {"name": "attn one token", "op": "attn", "lens": ",".join(["1"] * 16),
         "cols": "8192,7001,5120,4096,3333,2048,2048,1500,1024,777,512,300,129,64,33,1",
         "heads": 32, "kv_heads": 8, "dim": 128, "bias": "none", "causal": False,
         "layout": "split", "dtype": "bf16"},
        # Long packed sequences, causal, shared key heads, behind a fused projection.
        {"name": "attn long causal", "op": "attn", "lens": "6000,4097,1500,257", "cols": "",
         "heads": 16, "kv_heads": 4, "dim": 128, "bias": "none", "causal": True,
         "layout": "fused", "dtype": "bf16"},
        # The training step of the long square batch: bias and its gradient.
        {"name": "attn_bwd long_square", "op": "attn_bwd", "lens": "1024,768,384,96", "cols": "",
         "heads": 12, "kv_heads": 12, "dim": 32, "bias": "plain", "causal": False,
         "layout": "split", "dtype": "bf16"},
        # The training step of long causal sequences with shared key heads.
        {"name": "attn_bwd causal", "op": "attn_bwd", "lens": "4096,2500,1111,300", "cols": "",
         "heads": 16, "kv_heads": 8, "dim": 64, "bias": "none", "causal": True,
         "layout": "split", "dtype": "bf16"},
        # The weights of four blocks (c_s 384, c_z 128, hidden 512): many small tensors.
        {"name": "adamw four blocks", "op": "adamw",
         "sizes": ",".join(["49152,49152,65536,65536,49152"] * 4), "bits": 32, "dtype": "f32",
         "master": False},
        # Large bf16 tensors with an fp32 copy and states in 8 bits.
        {"name": "adamw large 8 bits", "op": "adamw", "sizes": "33554432,16777216,16777216,4194304,1001,7",
         "bits": 8, "dtype": "bf16", "master": True},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _lengths(rng, most_rows, longest, samples):
    n = _log_int(rng, 1, samples)
    top = _log_int(rng, 4, longest)
    low = _log_int(rng, 1, top)
    got = []
    for _ in range(n):
        x = _log_int(rng, low, top)
        if sum(got) + x <= most_rows:
            got.append(x)
    got = got or [top]
    if rng.random() < 0.2:
        got.insert(rng.randrange(len(got) + 1), 0)  # an empty sample
    return got


def _text(v):
    return ",".join(str(x) for x in v)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "attn", "attn", "attn_bwd", "attn_bwd", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "adamw":
        n = rng.randint(1, 10)
        sizes = [_log_int(rng, 1, 6_000_000) for _ in range(n)]
        return {"op": op, "sizes": _text(sizes), "bits": rng.choice([8, 32]), "dtype": dtype,
                "master": dtype == "bf16" and rng.random() < 0.5}
    dim = 8 * rng.randint(1, 16)
    group = rng.choice([1, 1, 2, 4])
    kv_heads = rng.randint(1, 8)
    heads = group * kv_heads
    if op in ("norm", "norm_bwd"):
        return {"op": op, "lens": _text(_lengths(rng, 16384, 8192, 16)), "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "rot": 2 * rng.randint(1, dim // 2),
                "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "parts"]),
                "layout": rng.choice(["split", "fused"]), "dtype": dtype,
                "offset": rng.random() < 0.3}
    lens = _lengths(rng, 4096, 2048, 12)
    case = {"op": op, "lens": _text(lens), "cols": "", "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "bias": rng.choice(["none", "plain", "masked"]),
            "causal": rng.random() < 0.4, "layout": rng.choice(["split", "fused"]),
            "dtype": dtype}
    if rng.random() < 0.3:  # queries of the rows over other columns
        cols = [_log_int(rng, 1, 4096) for _ in lens]
        if op == "attn" and rng.random() < 0.5:
            lens = [rng.randint(1, 4) for _ in lens]
        case.update(lens=_text(lens), cols=_text(cols), layout="split")
    widest = max(_ints(case["lens"])) * max(_ints(case["cols"] or case["lens"]))
    if len(lens) * heads * widest > 2.5e8:  # within the largest listed case
        case.update(heads=kv_heads)
    if len(lens) * case["heads"] * widest > 2.5e8:
        case.update(heads=1, kv_heads=1)
    return case


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _shape(case):
    rows = _ints(case["lens"])
    cols = _ints(case["cols"]) if case.get("cols") else rows
    return rows, cols


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# -------------------------------------------------------------------- inputs
def _normal(gen, shape, dtype=torch.float32, scale=1.0, mean=0.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale + mean).to(dtype)


def _heads_of(gen, case, rows, cols):
    """q, k, v: separate, or parts of one projected array."""
    T, Tc = sum(rows), sum(cols)
    H, K, D, dt = case["heads"], case["kv_heads"], case["dim"], _dtype(case)
    if case["layout"] == "fused":
        x = _normal(gen, (T, H + 2 * K, D), dt)
        return x[:, :H], x[:, H:H + K], x[:, H + K:]
    return _normal(gen, (T, H, D), dt), _normal(gen, (Tc, K, D), dt), _normal(gen, (Tc, K, D), dt)


def _frequencies(case):
    """Angles per position, in 64 bits, of the scaled rotation."""
    R, base, factor, original = case["rot"], 10000.0, 4.0, 2048.0
    f = base ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "parts":
        turns = original * f / (2.0 * math.pi)  # turns within the trained length
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _table(case, positions):
    """cos | sin of every position, the plan a program makes once."""
    f, magnitude = _frequencies(case)
    a = np.arange(positions, dtype=np.float64)[:, None] * f[None]
    both = np.concatenate([np.cos(a), np.sin(a)], 1) * magnitude
    return torch.from_numpy(both.astype(np.float32)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "adamw":
        return _prepare_adamw(case, gen)
    rows, cols = _shape(case)
    s = {"case": case, "rows": rows, "cols": cols}
    s["q"], s["k"], s["v"] = _heads_of(gen, case, rows, cols)
    dt, D = _dtype(case), case["dim"]
    if case["op"] in ("norm", "norm_bwd"):
        s["w_q"], s["w_k"] = (_normal(gen, (D,), scale=0.2, mean=1.0) for _ in range(2))
        longest = max(rows)
        start = torch.randint(0, 1000, (len(rows),), generator=gen, device="cuda")
        s["table"] = _table(case, longest + (1000 if case["offset"] else 0))
        s["positions"] = None
        if case["offset"]:  # every sample continues at a position of its own
            n = torch.tensor(rows, device="cuda")
            first = torch.cumsum(n, 0) - n
            at = torch.arange(sum(rows), device="cuda") - torch.repeat_interleave(first, n)
            s["positions"] = (at + torch.repeat_interleave(start, n)).to(torch.int32)
        if case["op"] == "norm_bwd":
            s["g_q"] = _normal(gen, tuple(s["q"].shape), dt)
            s["g_k"] = _normal(gen, tuple(s["k"].shape), dt)
    else:
        s["scale"] = 1.0 / math.sqrt(D)
        s["bias"] = None
        cells = sum(n * m for n, m in zip(rows, cols))
        if case["bias"] != "none":
            s["bias"] = _normal(gen, (case["heads"], cells), dt)
        if case["bias"] == "masked":  # cells left out, and one row left with nothing
            out = torch.rand((1, cells), generator=gen, device="cuda") < 0.1
            out[:, :next((m for n, m in zip(rows, cols) if n * m), 0)] = True
            s["bias"] = s["bias"].masked_fill(out, -math.inf)
        if case["op"] == "attn_bwd":
            s["g_o"] = _normal(gen, tuple(s["q"].shape), dt)
            s["o"], s["lse"] = _attention(s)
    if own:
        import padding_free_pair_amd as nt
        s["nt"] = nt
        s["partition"] = nt.nt_make_partition_rect(rows, cols) if case.get("cols") else \
            nt.nt_make_partition(rows)
    return s


def _prepare_adamw(case, gen):
    sizes, bits = _ints(case["sizes"]), case["bits"]
    s = {"case": case, "step": 10, "lr": 1e-3, "beta1": 0.9, "beta2": 0.99, "eps": 1e-8,
         "weight_decay": 0.01}
    full = [_normal(gen, (n,), scale=0.02) for n in sizes]
    s["params"] = [x.to(_dtype(case)) for x in full]
    s["masters"] = full if case["master"] else None
    s["grads"] = [_normal(gen, (n,), scale=1e-3) for n in sizes]
    m = [_normal(gen, (n,), scale=3e-4) for n in sizes]
    root = [_normal(gen, (n,), scale=3e-4).abs() + 1e-5 for n in sizes]
    if bits == 8:
        s["m"], s["m_scales"] = map(list, zip(*[_quantise(x) for x in m]))
        s["v"], s["v_scales"] = map(list, zip(*[_quantise(x, True) for x in root]))
    else:
        s["m"], s["v"] = m, [x * x for x in root]
        s["m_scales"] = s["v_scales"] = None
    if own:
        import padding_free_pair_amd as nt
        s["nt"] = nt
        s["tensors"] = nt.nt_adamw_tensors(s["params"], s["grads"], s["m"], s["v"],
                                           m_scales=s["m_scales"], v_scales=s["v_scales"],
                                           masters=s["masters"])
    return s


# --------------------------------------------------------------------- passes
def run(s):
    return {"norm": _run_norm, "norm_bwd": _run_norm_bwd, "attn": _run_attn,
            "attn_bwd": _run_attn_bwd, "adamw": _run_adamw}[s["case"]["op"]](s)


def _run_norm(s):
    if own:
        return s["nt"].nt_qk_norm_rotary(s["partition"], s["q"], s["k"], s["w_q"], s["w_k"],
                                         s["table"], interleaved=s["case"]["interleaved"],
                                         positions_q=s["positions"], positions_k=s["positions"])
    cos, sin = _angles(s)
    return tuple(_turn(_normed(x, w)[0], cos, sin, s["case"]).to(x.dtype)
                 for x, w in ((s["q"], s["w_q"]), (s["k"], s["w_k"])))


def _run_norm_bwd(s):
    if own:
        return s["nt"].nt_qk_norm_rotary_backward(
            s["partition"], s["q"], s["k"], s["g_q"], s["g_k"], s["w_q"], s["w_k"], s["table"],
            interleaved=s["case"]["interleaved"], positions_q=s["positions"],
            positions_k=s["positions"])
    cos, sin = _angles(s)
    (g_q, g_wq), (g_k, g_wk) = (_norm_bwd(x, g, w, cos, sin, s["case"]) for x, g, w in (
        (s["q"], s["g_q"], s["w_q"]), (s["k"], s["g_k"], s["w_k"])))
    return g_q, g_k, g_wq, g_wk


def _run_attn(s):
    if own:
        return s["nt"].nt_single_attention(s["partition"], s["q"], s["k"], s["v"], bias=s["bias"],
                                           causal=s["case"]["causal"], scale=s["scale"])
    return _attention(s)


def _run_attn_bwd(s):
    if own:
        return s["nt"].nt_single_attention_backward(
            s["partition"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["g_o"], bias=s["bias"],
            causal=s["case"]["causal"], scale=s["scale"])
    return _attention_bwd(s)


def _run_adamw(s):
    s["step"] += 1
    if own:
        s["nt"].nt_adamw_step(s["tensors"], step=s["step"], lr=s["lr"], beta1=s["beta1"],
                              beta2=s["beta2"], eps=s["eps"], weight_decay=s["weight_decay"])
    else:
        [_adamw(s, i) for i in range(len(s["params"]))]
    return {k: s[k] for k in ("params", "masters", "m", "v", "m_scales", "v_scales")}


# ----------------------------------------------------------- plain: the norm
def _angles(s):
    R = s["case"]["rot"]
    at = s["positions"]
    if at is None:
        n = torch.tensor(s["rows"], device="cuda")
        first = torch.cumsum(n, 0) - n
        at = torch.arange(sum(s["rows"]), device="cuda") - torch.repeat_interleave(first, n)
    row = s["table"][at.long()][:, None]
    return row[..., :R // 2], row[..., R // 2:]


def _pairs(x, case):
    R = case["rot"]
    if case["interleaved"]:
        return x[..., 0:R:2], x[..., 1:R:2]
    return x[..., :R // 2], x[..., R // 2:R]


def _joined(a, b, rest, case):
    if case["interleaved"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _turn(x, cos, sin, case):
    a, b = _pairs(x, case)
    return _joined(a * cos - b * sin, b * cos + a * sin, x[..., case["rot"]:], case)


def _normed(x, w):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    return x * r * w, x * r, r


def _norm_bwd(x, g, w, cos, sin, case):
    _, xhat, r = _normed(x, w)
    g = _turn(g.float(), cos, -sin, case)
    g_w = (g * xhat).sum((0, 1), dtype=torch.float64).float()
    g = g * w
    return ((g - xhat * (g * xhat).mean(-1, keepdim=True)) * r).to(x.dtype), g_w


# ------------------------------------------------------ plain: the attention
def _places(s):
    """Padded places: row and column singles, cells, and which hold something."""
    n, m = (torch.tensor(x, device="cuda") for x in (s["rows"], s["cols"]))
    r = torch.arange(max(s["rows"]), device="cuda")
    c = torch.arange(max(s["cols"]), device="cuda")
    eta, mu, o = (torch.cumsum(x, 0) - x for x in (n, m, n * m))
    in_r, in_c = r < n[:, None], c < m[:, None]
    at_r = torch.where(in_r, eta[:, None] + r, 0)
    at_c = torch.where(in_c, mu[:, None] + c, 0)
    seen = in_r[:, :, None] & in_c[:, None, :]
    cell = torch.where(seen, o[:, None, None] + r[:, None] * m[:, None, None] + c, 0)
    live = seen
    if s["case"]["causal"]:
        live = seen & (c <= r[:, None] + (m - n)[:, None, None])
    return at_r, at_c, in_r, in_c, cell, seen, live


def _padded(x, at, inside, heads):
    """[B, heads, N, D] in fp32 of packed [T, h, D]; shared heads repeated."""
    x = x.float()[at] * inside[:, :, None, None]
    x = x.permute(0, 2, 1, 3)
    return x.repeat_interleave(heads // x.shape[1], 1).contiguous()


def _scores(s, q, k, place):
    at_r, at_c, in_r, in_c, cell, seen, live = place
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()) * s["scale"]
    if s["bias"] is not None:
        x = x + s["bias"].float()[:, cell].transpose(0, 1)
    return x.masked_fill(~live[:, None], -math.inf)


def _attention(s):
    place = _places(s)
    at_r, at_c, in_r, in_c = place[:4]
    H = s["case"]["heads"]
    q, k, v = (_padded(x, a, i, H) for x, a, i in (
        (s["q"], at_r, in_r), (s["k"], at_c, in_c), (s["v"], at_c, in_c)))
    x = _scores(s, q, k, place)
    most = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(most), 0.0, most))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = (most + torch.log(total)).squeeze(-1)
    return o.transpose(1, 2)[in_r].to(s["q"].dtype), lse.transpose(1, 2)[in_r]


def _attention_bwd(s):
    place = _places(s)
    at_r, at_c, in_r, in_c, cell, seen, live = place
    H, K = s["case"]["heads"], s["case"]["kv_heads"]
    dt = s["q"].dtype
    q, o, g = (_padded(x, at_r, in_r, H) for x in (s["q"], s["o"], s["g_o"]))
    k, v = (_padded(x, at_c, in_c, H) for x in (s["k"], s["v"]))
    lse = s["lse"][at_r].permute(0, 2, 1)[..., None]
    p = torch.exp(_scores(s, q, k, place) - torch.where(torch.isinf(lse), 0.0, lse))
    ds = torch.matmul(g, v.transpose(-1, -2).contiguous())
    ds = p * (ds - (g * o).sum(-1, keepdim=True))
    g_v = torch.matmul(p.transpose(-1, -2).contiguous(), g)
    g_k = torch.matmul(ds.transpose(-1, -2).contiguous(), q) * s["scale"]
    g_q = torch.matmul(ds, k) * s["scale"]
    g_k, g_v = (x.unflatten(1, (K, H // K)).sum(2).transpose(1, 2)[in_c].to(dt)
                for x in (g_k, g_v))
    g_bias = None if s["bias"] is None else ds.transpose(0, 1)[:, seen].to(dt)
    return g_q.transpose(1, 2)[in_r].to(dt), g_k, g_v, g_bias


# ---------------------------------------------------------- plain: the update
def _blocks(x):
    n = x.numel()
    return torch.nn.functional.pad(x, (0, -n % STATE_BLOCK)).view(-1, STATE_BLOCK)


def _quantise(x, positive=False):
    """e4m3 codes and their scales, one for each 256 elements."""
    b = _blocks(x)
    scale = b.abs().amax(1) / E4M3_MAX
    y = b / torch.where(scale == 0, 1.0, scale)[:, None]
    if positive:
        y = torch.where(y > 0, y.clamp(min=E4M3_LEAST), y)
    return y.to(torch.float8_e4m3fn).view(-1)[:x.numel()].clone(), scale


def _values(codes, scale):
    n = codes.numel()
    return (_blocks(codes.float()) * scale[:, None]).view(-1)[:n]


def _adamw(s, i):
    eight = s["case"]["bits"] == 8
    g = s["grads"][i]
    p = (s["masters"][i] if s["masters"] else s["params"][i]).float()
    m = _values(s["m"][i], s["m_scales"][i]) if eight else s["m"][i]
    v = _values(s["v"][i], s["v_scales"][i]).square() if eight else s["v"][i]
    m = s["beta1"] * m + (1.0 - s["beta1"]) * g
    v = s["beta2"] * v + (1.0 - s["beta2"]) * g * g
    c1, c2 = 1.0 - s["beta1"] ** s["step"], 1.0 - s["beta2"] ** s["step"]
    p = p * (1.0 - s["lr"] * s["weight_decay"]) - \
        s["lr"] * (m / c1) / (torch.sqrt(v / c2) + s["eps"])
    if s["masters"]:
        s["masters"][i].copy_(p)
    s["params"][i].copy_(p)
    if eight:
        for name, x, positive in (("m", m, False), ("v", torch.sqrt(v), True)):
            codes, scale = _quantise(x, positive)
            s[name][i].copy_(codes)
            s[name + "_scales"][i].copy_(scale)
    else:
        s["m"][i].copy_(m)
        s["v"][i].copy_(v)


# ----------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "adamw":
        n = sum(_ints(case["sizes"]))
        state = 2 * (1 + 4 / STATE_BLOCK) if case["bits"] == 8 else 8
        full = 8 if case["master"] else 0
        param = e if case["master"] else 2 * e  # with a full copy the parameter is written only
        return {"bytes": n * (4 + param + full + 2 * state), "flops": 15 * n}
    rows, cols = _shape(case)
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    q, k = sum(rows) * H * D, sum(cols) * K * D
    if case["op"] in ("norm", "norm_bwd"):
        pos = 4 * sum(rows) if case["offset"] else 0
        table = 4 * case["rot"] * max(rows)
        if case["op"] == "norm":
            return {"bytes": 2 * e * (q + k) + table + pos + 8 * D, "flops": 8 * (q + k)}
        return {"bytes": 3 * e * (q + k) + table + pos + 16 * D, "flops": 16 * (q + k)}
    cells = sum(n * m for n, m in zip(rows, cols))
    live = cells
    if case["causal"]:
        live = sum(sum(max(0, min(m, r + 1 + m - n)) for r in range(n)) for n, m in zip(rows, cols))
    bias = 0 if case["bias"] == "none" else e * H * cells
    lse = 4 * sum(rows) * H
    if case["op"] == "attn":
        return {"bytes": e * (2 * q + 2 * k) + bias + lse, "flops": 4 * D * H * live}
    return {"bytes": e * (4 * q + 4 * k) + 2 * bias + lse, "flops": 10 * D * H * live}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm, "attn": _exact_attn,
            "attn_bwd": _exact_attn, "adamw": _exact_adamw}[case["op"]](s)


def _exact_norm(s):
    case, rows = s["case"], s["rows"]
    R = case["rot"]
    at = s["positions"] if s["positions"] is not None else \
        torch.cat([torch.arange(n, device="cuda") for n in rows])
    table = s["table"].double()[at.long()]
    # the rotation as complex numbers: (a + i b) (cos + i sin)
    unit = torch.complex(table[:, :R // 2], table[:, R // 2:])[:, None]

    def rotate(y, u):
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if case["interleaved"] else \
            (y[..., :R // 2], y[..., R // 2:R])
        t = torch.complex(a, b) * u
        out = y.clone()
        if case["interleaved"]:
            out[..., 0:R:2], out[..., 1:R:2] = t.real, t.imag
        else:
            out[..., :R // 2], out[..., R // 2:R] = t.real, t.imag
        return out

    outs = []
    for x, w, g in ((s["q"], s["w_q"], s.get("g_q")), (s["k"], s["w_k"], s.get("g_k"))):
        x, w = x.double(), w.double()
        rms = (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + 1e-6).sqrt()
        if g is None:
            outs.append(rotate(x / rms * w, unit))
        else:
            h = rotate(g.double(), unit.conj())
            hw = h * w
            dot = (hw * x).sum(-1, keepdim=True)
            outs.append((hw / rms - x * dot / (x.shape[-1] * rms ** 3), (h * x / rms).sum((0, 1))))
    if "g_q" not in s:
        return tuple(outs)
    (g_q, g_wq), (g_k, g_wk) = outs
    return g_q, g_k, g_wq, g_wk


def _exact_attn(s):
    case, rows, cols = s["case"], s["rows"], s["cols"]
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    back = case["op"] == "attn_bwd"
    G = H // K
    new = lambda t: torch.zeros(tuple(t.shape), dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = new(s["q"]), torch.zeros((sum(rows), H), dtype=torch.float64, device="cuda")
    g_q, g_k, g_v = new(s["q"]), new(s["k"]), new(s["v"])
    g_b = None if s["bias"] is None else new(s["bias"])
    a = b = cell = 0
    for n, m in zip(rows, cols):
        if n:
            hidden = torch.zeros((n, m), dtype=torch.bool, device="cuda")
            if case["causal"]:
                hidden = torch.ones((n, m), dtype=torch.bool, device="cuda").triu(m - n + 1)
            for h in range(H):
                q, k, v = s["q"][a:a + n, h].double(), s["k"][b:b + m, h // G].double(), \
                    s["v"][b:b + m, h // G].double()
                x = s["scale"] * (q @ k.T.contiguous())
                if s["bias"] is not None:
                    x = x + s["bias"][h, cell:cell + n * m].view(n, m).double()
                x = x.masked_fill(hidden, -math.inf)
                if not back:
                    lse[a:a + n, h] = torch.logsumexp(x, -1) if m else -math.inf
                    p = torch.exp(x - lse[a:a + n, h, None]).nan_to_num(0.0)
                    o[a:a + n, h] = p @ v
                    continue
                z = s["lse"][a:a + n, h, None].double()
                p = torch.where(torch.isinf(z), 0.0, torch.exp(x - z))
                g = s["g_o"][a:a + n, h].double()
                d = p * (g @ v.T.contiguous() - (g * s["o"][a:a + n, h].double()).sum(1)[:, None])
                d = torch.where(p == 0, 0.0, d)
                g_q[a:a + n, h] = s["scale"] * (d @ k)
                g_k[b:b + m, h // G] += s["scale"] * (d.T.contiguous() @ q)
                g_v[b:b + m, h // G] += p.T.contiguous() @ g
                if g_b is not None:
                    g_b[h, cell:cell + n * m] = d.reshape(-1)
        a, b, cell = a + n, b + m, cell + n * m
    return (g_q, g_k, g_v, g_b) if back else (o, lse)


def _exact_adamw(s):
    t, b1, b2, lr = s["step"] + 1, s["beta1"], s["beta2"], s["lr"]
    out = {k: [] for k in ("params", "masters", "m", "v", "m_scales", "v_scales")}
    for i, g in enumerate(s["grads"]):
        g, n = g.double(), g.numel()
        m, v = s["m"][i].double(), s["v"][i].double()
        which = torch.arange(n, device="cuda") // STATE_BLOCK
        if s["m_scales"]:
            m = m * s["m_scales"][i].double()[which]
            v = (v * s["v_scales"][i].double()[which]) ** 2
        m, v = m + (1 - b1) * (g - m), v + (1 - b2) * (g * g - v)
        p = (s["masters"][i] if s["masters"] else s["params"][i]).double()
        step = m / (1 - b1 ** t) / ((v / (1 - b2 ** t)) ** 0.5 + s["eps"])
        p = p - lr * (step + s["weight_decay"] * p)
        out["params"].append(p)
        out["masters"].append(p)
        if s["m_scales"]:  # the states in units of their block's scale, before the codes' rounding
            for name, x in (("m", m), ("v", v ** 0.5)):
                top = torch.zeros(s[name + "_scales"][i].numel(), dtype=torch.float64, device="cuda")
                top = top.scatter_reduce(0, which, x.abs(), "amax") / E4M3_MAX
                out[name].append(x / top[which])
                out[name + "_scales"].append(top)
        else:
            out["m"].append(m)
            out["v"].append(v)
    return {k: v if s[k] is not None else None for k, v in out.items()}
