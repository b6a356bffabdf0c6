"""Cases of the operators between tokens and singles, and of the singles' norm.

The operators: the embedding of tokens as singles with its gradient, the norm
of singles with the residual's addition (in the storage type or in 8 bits)
with its gradient, and the cross entropy of singles over a vocabulary with its
gradients. `run` computes them in plain torch or, where `own` is true, through
the library.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0  # largest finite e4m3 value
EPS = 1e-6


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One new token of each of sixteen samples: the latency of a lookup.
        {"name": "embed one token", "op": "embed", "tokens": 16, "rows": 32000, "width": 2048,
         "dtype": "bf16", "ids": "flat", "absent": 0.0, "scale": 1.0},
        # A long packed batch over a large vocabulary, scaled by the root of the width.
        {"name": "embed long", "op": "embed", "tokens": 16384, "rows": 128000, "width": 2048,
         "dtype": "bf16", "ids": "natural", "absent": 0.0, "scale": math.sqrt(2048.0)},
        # The long square batch over an alphabet of residues: few tokens, each many times.
        {"name": "embed_bwd alphabet", "op": "embed_bwd", "tokens": 2272, "rows": 33, "width": 384,
         "dtype": "f32", "ids": "flat", "absent": 0.1, "scale": 1.0, "accumulate": False},
        # A long packed batch over a vocabulary of odd size: some tokens often, most never.
        {"name": "embed_bwd long", "op": "embed_bwd", "tokens": 16384, "rows": 50021,
         "width": 1024, "dtype": "bf16", "ids": "natural", "absent": 0.0, "scale": 32.0,
         "accumulate": False},
        # One new token of each of sixteen samples, for a projection in 8 bits.
        {"name": "norm one token", "op": "norm", "tokens": 16, "width": 4096, "dtype": "bf16",
         "residual": True, "out": "row8"},
        # A long packed batch, 8 bits with a scale for every 128 values.
        {"name": "norm long", "op": "norm", "tokens": 16384, "width": 4096, "dtype": "bf16",
         "residual": True, "out": "group8"},
        # The high-variation batch trained in fp32, c_s 384.
        {"name": "norm_bwd high_variation", "op": "norm_bwd", "tokens": 1866, "width": 384,
         "dtype": "f32", "residual": False},
        # A long packed batch with wide singles, the residual's gradient joining.
        {"name": "norm_bwd long", "op": "norm_bwd", "tokens": 16384, "width": 4096,
         "dtype": "bf16", "residual": True},
        # The log probability of one token of each of sixteen samples.
        {"name": "loss one token", "op": "loss", "tokens": 16, "rows": 32000, "width": 2048,
         "dtype": "bf16", "absent": 0.0, "scale": 1.0},
        # Evaluation of a long packed batch over a large vocabulary of odd size.
        {"name": "loss long", "op": "loss", "tokens": 8007, "rows": 65537, "width": 2048,
         "dtype": "bf16", "absent": 0.0, "scale": 1.0},
        # The high-variation batch in fp32, half of its tokens hidden and predicted.
        {"name": "loss_bwd high_variation", "op": "loss_bwd", "tokens": 1866, "rows": 4099,
         "width": 384, "dtype": "f32", "absent": 0.5, "scale": 1.0, "both": False,
         "accumulate": False},
        # The training step of a long packed batch, with a term in the log sum squared.
        {"name": "loss_bwd long", "op": "loss_bwd", "tokens": 8007, "rows": 32003, "width": 2048,
         "dtype": "bf16", "absent": 0.0, "scale": 1.0, "both": True, "accumulate": False},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["embed", "embed_bwd", "norm", "norm_bwd", "loss", "loss_bwd"])
    case = {"op": op, "tokens": _log_int(rng, 1, 16384), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op in ("norm", "norm_bwd"):
        case["width"] = 8 * _log_int(rng, 1, 1024)
        case["tokens"] = max(1, min(case["tokens"], 16384 * 4096 // case["width"]))
        case["residual"] = rng.random() < 0.6
        if op == "norm":
            case["out"] = rng.choice(["same", "row8", "group8"])
            if case["out"] == "group8":
                case["width"] = max(128, case["width"] // 128 * 128)
        return case
    case["rows"] = _log_int(rng, 2, 131072)
    case["absent"] = rng.choice([0.0, 0.0, 0.15, 0.85])
    if op in ("embed", "embed_bwd"):
        case["width"] = 8 * _log_int(rng, 1, 256)
        case["ids"] = rng.choice(["flat", "natural"])
        case["scale"] = rng.choice([1.0, math.sqrt(case["width"])])
        if op == "embed_bwd":
            case["accumulate"] = rng.random() < 0.3
            case["rows"] = max(2, min(case["rows"], 50021 * 1024 // case["width"]))
        return case
    case["width"] = 8 * _log_int(rng, 4, 256)
    case["scale"] = rng.choice([1.0, 1.0, 0.25])
    most = 1.0e12 if op == "loss" else 5.0e11  # within the largest listed case
    case["rows"] = max(2, min(case["rows"], int(most / (case["tokens"] * case["width"]))))
    if op == "loss_bwd":
        case["both"] = rng.random() < 0.5
        case["accumulate"] = rng.random() < 0.3
    return case


# -------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(gen, shape, dtype=torch.float32, scale=1.0, mean=0.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale + mean).to(dtype)


def _absent(case):
    return int(round(case["tokens"] * case["absent"]))


def _ids(gen, case, kind):
    """Tokens; as many as the case says are absent (-1), at places of the seed."""
    u = torch.rand(case["tokens"], generator=gen, device="cuda", dtype=torch.float64)
    V = case["rows"]
    # "natural": the k-th most frequent token about 1 / k as often as the first
    x = torch.exp(u * math.log(V + 1.0)) - 1.0 if kind == "natural" else u * V
    ids = x.floor().clamp(max=V - 1).to(torch.int32)
    ids[torch.randperm(case["tokens"], generator=gen, device="cuda")[:_absent(case)]] = -1
    return ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    op, T, C, dt = case["op"], case["tokens"], case["width"], _dtype(case)
    if op in ("norm", "norm_bwd"):
        s["w"] = _normal(gen, (C,), scale=0.2, mean=1.0)
        if op == "norm":
            s["x"] = _normal(gen, (T, C), dt)
            s["residual"] = _normal(gen, (T, C), dt, 2.0) if case["residual"] else None
        else:
            s["h"] = _normal(gen, (T, C), dt, 2.0)
            s["g_y"] = _normal(gen, (T, C), dt)
            s["g_h"] = _normal(gen, (T, C), dt) if case["residual"] else None
        return s
    V = case["rows"]
    s["ids"] = _ids(gen, case, case.get("ids", "natural"))
    if op == "embed":
        s["table"] = _normal(gen, (V, C), dt, 0.02)
    elif op == "embed_bwd":
        s["g"] = _normal(gen, (T, C), dt)
    else:
        s["x"] = _normal(gen, (T, C), dt)
        s["W"] = _normal(gen, (V, C), dt, 2.0 / math.sqrt(C))
        if op == "loss_bwd":
            s["lse"] = _loss(s)[1]
            n = max(1, T - _absent(case))
            s["g_nll"] = torch.full((T,), 1.0 / n, device="cuda")
            s["g_lse"] = s["lse"] * (2e-2 / n) if case["both"] else None
    if case.get("accumulate"):
        s["g_table"] = _normal(gen, (V, C), scale=1e-2)
    else:
        s["g_table"] = None
    return s


# --------------------------------------------------------------------- passes
def run(s):
    return {"embed": _run_embed, "embed_bwd": _run_embed_bwd, "norm": _run_norm,
            "norm_bwd": _run_norm_bwd, "loss": _run_loss, "loss_bwd": _run_loss_bwd}[
                s["case"]["op"]](s)


def _run_embed(s):
    if own:
        import padding_free_pair_amd as nt
        return nt.nt_token_embedding(s["table"], s["ids"], scale=s["case"]["scale"])
    out = s["table"][s["ids"].clamp(min=0).long()].float() * s["case"]["scale"]
    return (out * (s["ids"] >= 0)[:, None]).to(s["table"].dtype)


def _run_embed_bwd(s):
    case = s["case"]
    if own:
        import padding_free_pair_amd as nt
        return nt.nt_token_embedding_backward(s["ids"], s["g"], case["rows"], scale=case["scale"],
                                              g_table=s["g_table"], accumulate=case["accumulate"])
    g = s["g_table"]
    if g is None:
        g = torch.zeros((case["rows"], case["width"]), device="cuda")
    add = s["g"].float() * (case["scale"] * (s["ids"] >= 0)[:, None])
    return g.index_add_(0, s["ids"].clamp(min=0).long(), add)


def _run_norm(s):
    out = s["case"]["out"]
    if own:
        import padding_free_pair_amd as nt
        if out == "same":
            return nt.nt_residual_norm(s["x"], s["w"], residual=s["residual"], eps=EPS)
        return nt.nt_residual_norm_8bit(s["x"], s["w"], residual=s["residual"], eps=EPS,
                                        group=0 if out == "row8" else 128)
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(h.dtype)
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * s["w"]
    if out == "same":
        return y.to(h.dtype), h
    pieces = y.view(y.shape[0], -1, y.shape[1] if out == "row8" else 128)
    scales = pieces.abs().amax(2) / E4M3_MAX
    codes = pieces / torch.where(scales == 0, 1.0, scales)[:, :, None]
    return codes.to(torch.float8_e4m3fn).view(y.shape), scales, h


def _run_norm_bwd(s):
    if own:
        import padding_free_pair_amd as nt
        return nt.nt_residual_norm_backward(s["h"], s["g_y"], s["w"], g_h=s["g_h"], eps=EPS)
    f, g = s["h"].float(), s["g_y"].float()
    r = torch.rsqrt(f.square().mean(1, keepdim=True) + EPS)
    xhat = f * r
    g_w = (g * xhat).sum(0, dtype=torch.float64).float()
    g = g * s["w"]
    g = (g - xhat * (g * xhat).mean(1, keepdim=True)) * r
    if s["g_h"] is not None:
        g = g + s["g_h"].float()
    return g.to(s["h"].dtype), g_w


def _run_loss(s):
    if own:
        import padding_free_pair_amd as nt
        return nt.nt_token_loss(s["x"], s["W"], s["ids"], scale=s["case"]["scale"])
    return _loss(s)


def _logits(s):
    return (s["x"].float() @ s["W"].float().t()) * s["case"]["scale"]


def _loss(s):
    x = _logits(s)
    most = x.amax(1)
    lse = most + torch.log(torch.exp(x - most[:, None]).sum(1))
    at = x.gather(1, s["ids"].clamp(min=0).long()[:, None])[:, 0]
    live = s["ids"] >= 0
    return torch.where(live, lse - at, 0.0), torch.where(live, lse, 0.0)


def _run_loss_bwd(s):
    case = s["case"]
    if own:
        import padding_free_pair_amd as nt
        return nt.nt_token_loss_backward(s["x"], s["W"], s["ids"], s["lse"], s["g_nll"],
                                         g_lse=s["g_lse"], scale=case["scale"],
                                         g_W=s["g_table"], accumulate=case["accumulate"])
    live = (s["ids"] >= 0).float()
    g_nll = s["g_nll"] * live
    both = g_nll if s["g_lse"] is None else g_nll + s["g_lse"] * live
    d = torch.exp(_logits(s) - s["lse"][:, None]) * both[:, None]
    d.scatter_add_(1, s["ids"].clamp(min=0).long()[:, None], -g_nll[:, None])
    d *= case["scale"]
    g_x = (d @ s["W"].float()).to(s["x"].dtype)
    g_W = d.t() @ s["x"].float()
    return g_x, g_W if s["g_table"] is None else s["g_table"].add_(g_W)


# ----------------------------------------------------------------------- work
def _distinct(case):
    """How many tokens of the vocabulary a batch of the case's kind holds."""
    V, n = case["rows"], case["tokens"] - _absent(case)
    k = np.arange(V, dtype=np.float64)
    p = np.log((k + 2.0) / (k + 1.0)) / math.log(V + 1.0) if case["ids"] == "natural" else \
        np.full(V, 1.0 / V)
    return float((1.0 - (1.0 - p) ** n).sum())


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, T, C = case["op"], case["tokens"], case["width"]
    if op == "norm":
        read = e * T * C * (2 if case["residual"] else 1) + 4 * C
        write = T * C * e if case["out"] == "same" else \
            T * C + 4 * T * (1 if case["out"] == "row8" else C // 128)
        return {"bytes": read + write + (e * T * C if case["residual"] else 0), "flops": 6 * T * C}
    if op == "norm_bwd":
        return {"bytes": e * T * C * (4 if case["residual"] else 3) + 8 * C, "flops": 12 * T * C}
    V, live = case["rows"], T - _absent(case)
    if op == "embed":
        return {"bytes": 4 * T + e * C * (min(_distinct(case), live) + T), "flops": T * C}
    if op == "embed_bwd":
        table = 8 * _distinct(case) if case["accumulate"] else 4 * V
        return {"bytes": 4 * T + e * live * C + table * C, "flops": 2 * live * C}
    if op == "loss":
        return {"bytes": e * C * (live + V) + 12 * T, "flops": 2 * live * V * C}
    return {"bytes": e * C * (live + T + V) + 4 * V * C * (2 if case["accumulate"] else 1) + 16 * T,
            "flops": 6 * live * V * C}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "embed_bwd": _exact_embed_bwd, "norm": _exact_norm,
            "norm_bwd": _exact_norm, "loss": _exact_loss, "loss_bwd": _exact_loss}[case["op"]](s)


def _exact_embed(s):
    out = torch.zeros((s["ids"].numel(), s["table"].shape[1]), dtype=torch.float64, device="cuda")
    there = torch.nonzero(s["ids"] >= 0)[:, 0]
    out[there] = s["case"]["scale"] * s["table"].double()[s["ids"][there].long()]
    return out


def _exact_embed_bwd(s):
    """Sums of runs of equal tokens as differences of a running sum."""
    case = s["case"]
    out = torch.zeros((case["rows"], case["width"]), dtype=torch.float64, device="cuda")
    if s["g_table"] is not None:
        out += s["g_table"].double()
    there = torch.nonzero(s["ids"] >= 0)[:, 0]
    if there.numel() == 0:
        return out
    ids, order = torch.sort(s["ids"][there].long())
    total = torch.cumsum(s["g"][there[order]].double(), 0)
    last = torch.nonzero(torch.cat([ids[1:] != ids[:-1], torch.ones_like(ids[:1], dtype=torch.bool)]))
    ends = total[last[:, 0]]
    out[ids[last[:, 0]]] += case["scale"] * torch.diff(ends, dim=0, prepend=torch.zeros_like(ends[:1]))
    return out


def _exact_norm(s):
    case, w = s["case"], s["w"].double()
    if case["op"] == "norm":
        sums = s["x"].double() + (0.0 if s["residual"] is None else s["residual"].double())
        h = sums.to(s["x"].dtype).double()  # the norm is that of the stored sum
    else:
        h = s["h"].double()
    rms = (torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + EPS).sqrt()
    if case["op"] == "norm_bwd":
        g = s["g_y"].double()
        out = g * w / rms - h * (g * w * h).sum(1, keepdim=True) / (h.shape[1] * rms ** 3)
        if s["g_h"] is not None:
            out = out + s["g_h"].double()
        return out, (g * h / rms).sum(0)
    y = h / rms * w
    if case["out"] == "same":
        return y, sums
    n = h.shape[1] if case["out"] == "row8" else 128
    which = torch.arange(h.shape[1], device="cuda") // n
    top = torch.zeros((h.shape[0], h.shape[1] // n), dtype=torch.float64, device="cuda")
    top = top.index_reduce(1, which, y.abs(), "amax") / E4M3_MAX
    return y / top[:, which], top, sums  # the codes before their rounding


def _exact_loss(s):
    case = s["case"]
    there = torch.nonzero(s["ids"] >= 0)[:, 0]
    x, W, at = s["x"][there].double(), s["W"].double(), s["ids"][there].long()
    z = torch.mm(W, x.t().contiguous()) * case["scale"]  # [V, live]
    rows = torch.arange(there.numel(), device="cuda")
    if case["op"] == "loss":
        nll, lse = (torch.zeros(case["tokens"], dtype=torch.float64, device="cuda") for _ in "ab")
        lse[there] = torch.logsumexp(z, 0)
        nll[there] = lse[there] - z[at, rows]
        return nll, lse
    g_nll = s["g_nll"][there].double()
    g_lse = 0.0 if s["g_lse"] is None else s["g_lse"][there].double()
    z = (z - s["lse"][there].double()).exp_() * (g_nll + g_lse)
    z[at, rows] -= g_nll
    g_x = torch.zeros(tuple(s["x"].shape), dtype=torch.float64, device="cuda")
    g_x[there] = case["scale"] * torch.mm(z.t().contiguous(), W)
    g_W = case["scale"] * torch.mm(z, x)
    return g_x, g_W if s["g_table"] is None else s["g_table"].double() + g_W
