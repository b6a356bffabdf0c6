"""Binding of the single attention operators and of the optimizer's step.

Heads are [tokens, heads, head_dim] tensors whose heads are contiguous within
a token; the distance between tokens is free (a multiple of 8 elements), so
q, k and v may be parts of one projected tensor. As in the rest of the
binding, the functions check shapes and marshal pointers, and the library
computes.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

from . import Partition, _check, _code, _dtype_code, _native
from ._native import (NT_ADAMW_BLOCK, NT_OK, NT_ROTARY_LINEAR, NT_ROTARY_NONE, NT_ROTARY_PARTS,
                      NtAdamw, NtAdamwTensor, NtAttention, NtAttentionGrads, NtNormRotary,
                      NtRotary)

_SCALINGS = {"none": NT_ROTARY_NONE, "linear": NT_ROTARY_LINEAR, "parts": NT_ROTARY_PARTS}

# A call on a small batch takes a few microseconds on the GPU, so the host's
# part is kept as short: torch and the library are looked up once, and a
# tensor that is whole and contiguous passes its checks in one comparison.
_modules = None


def _load():
    global _modules
    if _modules is None:
        import torch
        _modules = torch, _native.lib()
    return _modules


class _Guard:
    """A call on a device that is not the current one, or on a given stream:
    outputs and workspaces that it allocates belong to that stream."""

    def __init__(self, torch, device, stream):
        self.torch, self.device, self.stream = torch, device, stream
        self.inner = torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)

    def __enter__(self) -> int:
        self.inner.__enter__()
        return (self.stream or self.torch.cuda.current_stream(self.device)).cuda_stream

    def __exit__(self, *exc):
        return self.inner.__exit__(*exc)


class _Here:
    """A call on the current device and its current stream."""

    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self) -> int:
        return self.handle

    def __exit__(self, *exc):
        return None


def _on(torch, device, stream):
    """The context of a call; yields the handle of the stream it launches on."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return _Here(torch._C._cuda_getCurrentRawStream(device.index))
        return _Guard(torch, device, None)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return _Guard(torch, device, stream)


def _heads(device, name, t, shape, dtype) -> int:
    """Checks a tensor of heads; returns the distance between its tokens."""
    tokens, heads, dim = shape
    if t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous():
        return heads * dim
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the partition on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.numel() == 0:
        return heads * dim
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != dim):
        raise ValueError(f"the heads of a token must be contiguous in {name}")
    if tokens == 1:
        return heads * dim
    if s[0] < heads * dim:
        raise ValueError(f"the tokens of {name} overlap")
    return s[0]


def _flat(device, name, t, shape, dtype) -> None:
    """Checks a contiguous tensor (None passes)."""
    if t is None or (t.shape == shape and t.dtype == dtype and t.device == device and
                     t.is_contiguous()):
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the partition on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} must be contiguous")


def _at(t) -> Optional[int]:
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _workspace(torch, device, workspace, need):
    """(pointer, bytes, the tensor that holds them) of a call's workspace."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, the partition on {device}")
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"workspace has {have} bytes, needs {need}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return _at(workspace), have, workspace


def nt_rotary_table(positions: int, rot_dim: int, base: float = 10000.0, scaling: str = "none",
                    factor: float = 1.0, original: float = 0.0, beta_fast: float = 32.0,
                    beta_slow: float = 1.0, magnitude: float = 1.0, device=None, stream=None):
    """The rotation's table, float32 [positions, rot_dim]: cosines, then sines.

    scaling: "none", "linear" (angles divided by factor) or "parts" (only
    the frequencies that turn seldom within `original` positions are
    divided; beta_fast and beta_slow are the turns between which the two
    blend). magnitude multiplies cosines and sines.
    """
    torch, lib = _load()
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    dev = torch.device(device) if device is not None else torch.device(
        "cuda", torch.cuda.current_device())
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    r = NtRotary(rot_dim, _SCALINGS[scaling], base, factor, original, beta_fast, beta_slow,
                 magnitude)
    with _on(torch, dev, stream) as s:
        table = torch.empty((positions, rot_dim), dtype=torch.float32, device=dev)
        _check(lib.nt_rotary_table(ctypes.byref(r), _at(table), positions, s))
    return table


def _norm_struct(torch, p, dev, q, k, w_q, w_k, table, interleaved, eps, positions_q, positions_k,
                 q_out, k_out):
    """The norm's description, with every tensor checked."""
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    T, heads, dim = p.T, q.shape[1], q.shape[2]
    dt, f32 = q.dtype, torch.float32
    ld_q = _heads(dev, "q", q, (T, heads, dim), dt)
    ld_qo = _heads(dev, "the output of q", q_out, (T, heads, dim), dt)
    kv = ld_k = ld_ko = 0
    if k is not None:
        kv, Tk = k.shape[1], p.T_cols
        ld_k = _heads(dev, "k", k, (Tk, kv, dim), dt)
        ld_ko = _heads(dev, "the output of k", k_out, (Tk, kv, dim), dt)
    rows = rot = 0
    if table is not None:
        if table.dim() != 2 or table.shape[1] == 0:
            raise ValueError("table must be [positions, rot_dim]")
        rows, rot = table.shape
        _flat(dev, "table", table, table.shape, f32)
    _flat(dev, "w_q", w_q, (dim,), f32)
    _flat(dev, "w_k", w_k, (dim,), f32)
    if positions_q is not None:
        _flat(dev, "positions_q", positions_q, (T,), torch.int32)
    if positions_k is not None:
        _flat(dev, "positions_k", positions_k, (p.T_cols,), torch.int32)
    return NtNormRotary(heads, kv, dim, rot, 1 if interleaved else 0, eps, rows, ld_q, ld_k, ld_qo,
                        ld_ko)


def nt_qk_norm_rotary(p: Partition, q, k=None, w_q=None, w_k=None, table=None,
                      interleaved: bool = False, eps: float = 1e-6, positions_q=None,
                      positions_k=None, q_out=None, k_out=None, stream=None):
    """Norm of every query and key head (w_q, w_k: float32 [head_dim]; None: no
    norm) and the rotation by the table's angles (None: no rotation), in one
    pass; returns (q_out, k_out). Positions are a token's index within its
    sample unless given (int32). q_out may be q and k_out k.
    """
    torch, lib = _load()
    code, dev = _dtype_code(q), p.device
    with _on(torch, dev, stream) as s:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k is None:
            k_out = None
        elif k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        n = _norm_struct(torch, p, dev, q, k, w_q, w_k, table, interleaved, eps, positions_q,
                         positions_k, q_out, k_out)
        status = lib.nt_qk_norm_rotary(
            ctypes.byref(p.struct), ctypes.byref(n), _at(q), _at(k), _at(w_q), _at(w_k),
            _at(table), _at(positions_q), _at(positions_k), _at(q_out), _at(k_out), code, s)
        if status != NT_OK:
            _check(status)
    return q_out, k_out


def _bytes(entry, p, a, code) -> int:
    b = ctypes.c_size_t()
    status = entry(ctypes.byref(p.struct), ctypes.byref(a), code, ctypes.byref(b))
    if status != NT_OK:
        _check(status)
    return b.value


def nt_qk_norm_rotary_backward_workspace_bytes(p: Partition, heads: int, kv_heads: int,
                                               head_dim: int, dtype) -> int:
    n = NtNormRotary(heads, kv_heads, head_dim, 0, 0, 0.0, 0, 0, 0, 0, 0)
    return _bytes(_native.lib().nt_qk_norm_rotary_backward_workspace_bytes, p, n, _code(dtype))


def nt_qk_norm_rotary_backward(p: Partition, q, k, g_q, g_k=None, w_q=None, w_k=None, table=None,
                               interleaved: bool = False, eps: float = 1e-6, positions_q=None,
                               positions_k=None, g_q_in=None, g_k_in=None, workspace=None,
                               stream=None):
    """Gradient of nt_qk_norm_rotary for the outputs' gradients g_q, g_k
    (contiguous); returns (g_q_in, g_k_in, g_w_q, g_w_k), the weights' in
    float32 (None without weights). g_q_in may be g_q and g_k_in g_k."""
    torch, lib = _load()
    code, dev, dt = _dtype_code(q), p.device, q.dtype
    with _on(torch, dev, stream) as s:
        if g_q_in is None:
            g_q_in = torch.empty(q.shape, dtype=dt, device=q.device)
        _flat(dev, "g_q", g_q, q.shape, dt)
        if k is None:
            g_k = g_k_in = w_k = None
        else:
            if g_k is None:
                raise ValueError("g_k is missing")
            if g_k_in is None:
                g_k_in = torch.empty(k.shape, dtype=dt, device=k.device)
            _flat(dev, "g_k", g_k, k.shape, dt)
        n = _norm_struct(torch, p, dev, q, k, w_q, w_k, table, interleaved, eps, positions_q,
                         positions_k, g_q_in, g_k_in)
        g_w_q = None if w_q is None else torch.empty_like(w_q)
        g_w_k = None if w_k is None else torch.empty_like(w_k)
        need = 0
        if w_q is not None or w_k is not None:
            need = _bytes(lib.nt_qk_norm_rotary_backward_workspace_bytes, p, n, code)
        ws, have, workspace = _workspace(torch, dev, workspace, need)
        status = lib.nt_qk_norm_rotary_backward(
            ctypes.byref(p.struct), ctypes.byref(n), _at(q), _at(k), _at(g_q), _at(g_k), _at(w_q),
            _at(w_k), _at(table), _at(positions_q), _at(positions_k), _at(g_q_in), _at(g_k_in),
            _at(g_w_q), _at(g_w_k), code, ws, have, s)
        if status != NT_OK:
            _check(status)
    return g_q_in, g_k_in, g_w_q, g_w_k


def _attention_struct(p, dev, q, k, v, causal, scale):
    """The attention's description, with q, k and v checked."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, head_dim]")
    heads, dim, kv, dt = q.shape[1], q.shape[2], k.shape[1], q.dtype
    if scale is None:
        scale = 1.0 / math.sqrt(dim) if dim else 1.0
    keys = (p.T_cols, kv, dim)
    return NtAttention(heads, kv, dim, 1 if causal else 0, scale,
                       _heads(dev, "q", q, (p.T, heads, dim), dt), _heads(dev, "k", k, keys, dt),
                       _heads(dev, "v", v, keys, dt))


def nt_attention_workspace_bytes(p: Partition, heads: int, kv_heads: int, head_dim: int,
                                 dtype, causal: bool = False) -> int:
    a = NtAttention(heads, kv_heads, head_dim, 1 if causal else 0, 1.0, 0, 0, 0)
    return _bytes(_native.lib().nt_attention_workspace_bytes, p, a, _code(dtype))


def nt_attention_backward_workspace_bytes(p: Partition, heads: int, kv_heads: int, head_dim: int,
                                          dtype, causal: bool = False) -> int:
    a = NtAttention(heads, kv_heads, head_dim, 1 if causal else 0, 1.0, 0, 0, 0)
    return _bytes(_native.lib().nt_attention_backward_workspace_bytes, p, a, _code(dtype))


def nt_single_attention(p: Partition, q, k, v, bias=None, causal: bool = False, scale=None,
                        o=None, lse=None, workspace=None, stream=None):
    """Attention of the row singles' queries q [T, heads, head_dim] over the
    column singles' keys and values [T_cols, kv_heads, head_dim] of the same
    sample, with a bias [heads, cells] from the pair state (-inf masks a
    cell) and, causal, without the keys past a query's place. scale defaults
    to 1 / sqrt(head_dim). Returns (o, lse), lse float32 [T, heads]."""
    torch, lib = _load()
    code, dev = _dtype_code(q), p.device
    with _on(torch, dev, stream) as s:
        a = _attention_struct(p, dev, q, k, v, causal, scale)
        rows = (p.T, a.heads)
        if o is None:
            o = torch.empty(q.shape, dtype=q.dtype, device=dev)
        else:
            _flat(dev, "o", o, q.shape, q.dtype)
        if lse is None:
            lse = torch.empty(rows, dtype=torch.float32, device=dev)
        else:
            _flat(dev, "lse", lse, rows, torch.float32)
        if bias is not None:
            _flat(dev, "bias", bias, (a.heads, p.cells), q.dtype)
        ws, have, workspace = _workspace(torch, dev, workspace,
                                         _bytes(lib.nt_attention_workspace_bytes, p, a, code))
        status = lib.nt_single_attention(ctypes.byref(p.struct), ctypes.byref(a), _at(q), _at(k),
                                         _at(v), _at(bias), _at(o), _at(lse), code, ws, have, s)
        if status != NT_OK:
            _check(status)
    return o, lse


def nt_single_attention_backward(p: Partition, q, k, v, o, lse, g_o, bias=None,
                                 causal: bool = False, scale=None, g_q=None, g_k=None, g_v=None,
                                 g_bias=None, bias_grad: bool = True, workspace=None,
                                 stream=None):
    """Gradients of nt_single_attention for g_o = dL/do (contiguous), from the
    forward's inputs, o and lse; returns (g_q, g_k, g_v, g_bias) in q's dtype
    (g_bias None without a bias, or with bias_grad False). g_q, g_k, g_v may
    be parts of one tensor, as q, k, v may."""
    torch, lib = _load()
    code, dev, dt = _dtype_code(q), p.device, q.dtype
    with _on(torch, dev, stream) as s:
        a = _attention_struct(p, dev, q, k, v, causal, scale)
        heads = a.heads
        _flat(dev, "o", o, q.shape, dt)
        _flat(dev, "g_o", g_o, q.shape, dt)
        _flat(dev, "lse", lse, (p.T, heads), torch.float32)
        if bias is None:
            if g_bias is not None:
                raise ValueError("g_bias without a bias")
        else:
            _flat(dev, "bias", bias, (heads, p.cells), dt)
            if g_bias is None and bias_grad:
                g_bias = torch.empty(bias.shape, dtype=dt, device=dev)
            _flat(dev, "g_bias", g_bias, (heads, p.cells), dt)
        ld = [a.heads * a.head_dim, a.kv_heads * a.head_dim, a.kv_heads * a.head_dim]
        out = [g_q, g_k, g_v]
        for i, (name, of) in enumerate((("g_q", q), ("g_k", k), ("g_v", v))):
            if out[i] is None:
                out[i] = torch.empty(of.shape, dtype=dt, device=dev)
            else:
                ld[i] = _heads(dev, name, out[i], tuple(of.shape), dt)
        g = NtAttentionGrads(_at(out[0]), _at(out[1]), _at(out[2]), _at(g_bias), *ld)
        ws, have, workspace = _workspace(
            torch, dev, workspace, _bytes(lib.nt_attention_backward_workspace_bytes, p, a, code))
        status = lib.nt_single_attention_backward(
            ctypes.byref(p.struct), ctypes.byref(a), _at(q), _at(k), _at(v), _at(bias), _at(o),
            _at(lse), _at(g_o), ctypes.byref(g), code, ws, have, s)
        if status != NT_OK:
            _check(status)
    return out[0], out[1], out[2], g_bias


class AdamwTensors:
    """Parameters with their gradients and states, checked and marshalled once
    (nt_adamw_tensors); nt_adamw_step updates them in place at every call."""

    def __init__(self, array, count, code, bits, device, keep):
        self.array, self.count, self.code, self.bits = array, count, code, bits
        self.device, self.keep = device, keep


def nt_adamw_states(params: Sequence, bits: int = 32):
    """States of a first step for nt_adamw_tensors: (m, v, m_scales,
    v_scales), zeros; in 8 bits m and v are float8_e4m3fn with one scale for
    each NT_ADAMW_BLOCK elements, else the scales are None."""
    torch = _load()[0]
    if bits not in (8, 32):
        raise ValueError("bits must be 32 or 8")
    dt = torch.float32 if bits == 32 else torch.float8_e4m3fn
    m, v = ([torch.zeros(p.shape, dtype=dt, device=p.device) for p in params] for _ in range(2))
    if bits == 32:
        return m, v, None, None
    ms, vs = ([torch.zeros(-(-p.numel() // NT_ADAMW_BLOCK), dtype=torch.float32, device=p.device)
               for p in params] for _ in range(2))
    return m, v, ms, vs


def nt_adamw_tensors(params: Sequence, grads: Sequence, m: Sequence, v: Sequence, m_scales=None,
                     v_scales=None, masters=None) -> AdamwTensors:
    """The tensors of nt_adamw_step: parameters (all bf16 or all fp32), fp32
    gradients, states as nt_adamw_states makes them and, optionally, fp32
    masters, the copies that are updated in bf16 parameters' place. The
    tensors are held, and their gradients read at every step, so gradients go
    into the same tensors each time."""
    torch = _load()[0]
    count = len(params)
    if count == 0:
        raise ValueError("at least one parameter")
    bits = 8 if m_scales is not None else 32
    if (m_scales is None) != (v_scales is None):
        raise ValueError("m_scales and v_scales go together")
    lists = {"grads": grads, "m": m, "v": v, "m_scales": m_scales, "v_scales": v_scales,
             "masters": masters}
    for name, x in lists.items():
        if x is not None and len(x) != count:
            raise ValueError(f"{name} has {len(x)} tensors, params {count}")
    dt, dev, f32 = params[0].dtype, params[0].device, torch.float32
    state = f32 if bits == 32 else torch.float8_e4m3fn
    array = (NtAdamwTensor * count)()
    for i, w in enumerate(params):
        scales = (-(-w.numel() // NT_ADAMW_BLOCK),)
        of = {"param": (w, w.shape, dt), "grad": (grads[i], w.shape, f32),
              "m": (m[i], w.shape, state), "v": (v[i], w.shape, state)}
        if masters is not None:
            of["master"] = (masters[i], w.shape, f32)
        if bits == 8:
            of["m_scale"] = (m_scales[i], scales, f32)
            of["v_scale"] = (v_scales[i], scales, f32)
        for name, (t, shape, want) in of.items():
            if t.device != dev:
                raise ValueError(f"{name} {i} is on {t.device}, the first parameter on {dev}")
            if tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name} {i} has shape {tuple(t.shape)}, expected {tuple(shape)}")
            if t.dtype != want:
                raise TypeError(f"{name} {i} has dtype {t.dtype}, expected {want}")
            if not t.is_contiguous():
                raise ValueError(f"{name} {i} must be contiguous")
            setattr(array[i], name, _at(t))
        array[i].n = w.numel()
    keep = [list(x) for x in (params, grads, m, v, m_scales, v_scales, masters) if x is not None]
    return AdamwTensors(array, count, _dtype_code(params[0]), bits, dev, keep)


def nt_adamw_step(tensors: AdamwTensors, step, lr=1e-3, beta1: float = 0.9, beta2: float = 0.999,
                  eps: float = 1e-8, weight_decay: float = 0.01, stream=None) -> None:
    """One AdamW step over the tensors, in place. step (1 for the first) and lr
    are numbers, or one-element device tensors (int64, float32) that the
    kernels read, so that a captured graph follows them."""
    torch, lib = _load()
    h = NtAdamw(0.0, beta1, beta2, eps, weight_decay, 0, None, None, tensors.bits)
    if isinstance(step, torch.Tensor):
        if step.dtype != torch.int64 or step.numel() != 1 or step.device != tensors.device:
            raise ValueError("a step tensor is one int64 on the parameters' device")
        h.step_device = step.data_ptr()
    else:
        h.step = step
    if isinstance(lr, torch.Tensor):
        if lr.dtype != torch.float32 or lr.numel() != 1 or lr.device != tensors.device:
            raise ValueError("an lr tensor is one float32 on the parameters' device")
        h.lr_device = lr.data_ptr()
    else:
        h.lr = lr
    with _on(torch, tensors.device, stream) as s:
        _check(lib.nt_adamw_step(tensors.array, tensors.count, ctypes.byref(h), tensors.code, s))
