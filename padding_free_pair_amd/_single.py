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

from . import (NtError, Partition, _check, _code, _dtype_code, _expect, _expect_workspace,  # noqa: F401
               _nbytes, _native, _torch)
from ._native import (NT_ADAMW_BLOCK, NT_ROTARY_LINEAR, NT_ROTARY_NONE, NT_ROTARY_PARTS,
                      NtAdamw, NtAdamwTensor, NtAttention, NtAttentionGrads, NtNormRotary,
                      NtRotary)

_SCALINGS = {"none": NT_ROTARY_NONE, "linear": NT_ROTARY_LINEAR, "parts": NT_ROTARY_PARTS}


class _On:
    """The device and stream of a call: outputs and workspaces that the call
    allocates belong to the stream that uses them. Yields the stream's handle."""

    __slots__ = ("device", "stream", "guard")

    def __init__(self, device, stream):
        self.device, self.stream, self.guard = device, stream, None

    def __enter__(self) -> int:
        torch = _torch()
        s = self.stream
        if s is None:
            if self.device.index != torch.cuda.current_device():
                self.guard = torch.cuda.device(self.device)
        else:
            if not hasattr(s, "cuda_stream"):
                s = torch.cuda.ExternalStream(int(s), device=self.device)
            self.guard = torch.cuda.stream(s)
        if self.guard is not None:
            self.guard.__enter__()
        return (s or torch.cuda.current_stream(self.device)).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _heads(p, name, t, tokens, heads, dim, dtype) -> int:
    """Checks a tensor of heads; returns the distance between its tokens."""
    if t.device != p.device:
        raise ValueError(f"{name} is on {t.device}, the partition on {p.device}")
    if t.shape != (tokens, heads, dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(tokens, heads, dim)}")
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


def _at(t) -> Optional[int]:
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _flat(p, name, t, shape, dtype) -> None:
    _expect(p, name, t, shape, dtype)
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def nt_rotary_table(positions: int, rot_dim: int, base: float = 10000.0, scaling: str = "none",
                    factor: float = 1.0, original: float = 0.0, beta_fast: float = 32.0,
                    beta_slow: float = 1.0, magnitude: float = 1.0, device=None, stream=None):
    """The rotation's table, float32 [positions, rot_dim]: cosines, then sines.

    scaling: "none", "linear" (angles divided by factor) or "parts" (only
    the frequencies that turn seldom within `original` positions are
    divided; beta_fast and beta_slow are the turns between which the two
    blend). magnitude multiplies cosines and sines.
    """
    torch = _torch()
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    dev = torch.device(device) if device is not None else torch.device(
        "cuda", torch.cuda.current_device())
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    r = NtRotary(rot_dim, _SCALINGS[scaling], base, factor, original, beta_fast, beta_slow,
                 magnitude)
    with _On(dev, stream) as s:
        table = torch.empty((positions, rot_dim), dtype=torch.float32, device=dev)
        _check(_native.lib().nt_rotary_table(ctypes.byref(r), _at(table), positions, s))
    return table


def _norm_struct(p, q, k, table, interleaved, eps, q_out, k_out):
    """The norm's description, with q, k and their counterparts checked."""
    torch = _torch()
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    heads, dim = q.shape[1], q.shape[2]
    kv = 0 if k is None else k.shape[1]
    n = NtNormRotary(heads, kv, dim, 0, 1 if interleaved else 0, eps, 0, 0, 0, 0, 0)
    n.ld_q = _heads(p, "q", q, p.T, heads, dim, q.dtype)
    n.ld_q_out = _heads(p, "the output of q", q_out, p.T, heads, dim, q.dtype)
    if k is not None:
        n.ld_k = _heads(p, "k", k, p.T_cols, kv, dim, q.dtype)
        n.ld_k_out = _heads(p, "the output of k", k_out, p.T_cols, kv, dim, q.dtype)
    if table is not None:
        if table.dim() != 2:
            raise ValueError("table must be [positions, rot_dim]")
        _flat(p, "table", table, tuple(table.shape), torch.float32)
        n.positions, n.rot_dim = table.shape
        if n.rot_dim == 0:
            raise ValueError("table rotates no dimension; pass table=None")
    return n


def _norm_inputs(p, dim, w_q, w_k, positions_q, positions_k):
    torch = _torch()
    _flat(p, "w_q", w_q, (dim,), torch.float32)
    _flat(p, "w_k", w_k, (dim,), torch.float32)
    _flat(p, "positions_q", positions_q, (p.T,), torch.int32)
    _flat(p, "positions_k", positions_k, (p.T_cols,), torch.int32)


def nt_qk_norm_rotary(p: Partition, q, k=None, w_q=None, w_k=None, table=None,
                      interleaved: bool = False, eps: float = 1e-6, positions_q=None,
                      positions_k=None, q_out=None, k_out=None, stream=None):
    """Norm of every query and key head (w_q, w_k: float32 [head_dim]; None: no
    norm) and the rotation by the table's angles (None: no rotation), in one
    pass; returns (q_out, k_out). Positions are a token's index within its
    sample unless given (int32). q_out may be q and k_out k.
    """
    torch = _torch()
    code = _dtype_code(q)
    with _On(p.device, stream) as s:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        n = _norm_struct(p, q, k, table, interleaved, eps, q_out, k_out)
        _norm_inputs(p, n.head_dim, w_q, w_k, positions_q, positions_k)
        _check(_native.lib().nt_qk_norm_rotary(
            ctypes.byref(p.struct), ctypes.byref(n), _at(q), _at(k), _at(w_q), _at(w_k),
            _at(table), _at(positions_q), _at(positions_k), _at(q_out),
            None if k is None else _at(k_out), code, s))
    return q_out, k_out if k is not None else None


def _norm_backward_bytes(p, n, code) -> int:
    b = ctypes.c_size_t()
    _check(_native.lib().nt_qk_norm_rotary_backward_workspace_bytes(
        ctypes.byref(p.struct), ctypes.byref(n), code, ctypes.byref(b)))
    return b.value


def nt_qk_norm_rotary_backward_workspace_bytes(p: Partition, heads: int, kv_heads: int,
                                               head_dim: int, dtype) -> int:
    n = NtNormRotary(heads, kv_heads, head_dim, 0, 0, 0.0, 0, 0, 0, 0, 0)
    return _norm_backward_bytes(p, n, _code(dtype))


def nt_qk_norm_rotary_backward(p: Partition, q, k, g_q, g_k=None, w_q=None, w_k=None, table=None,
                               interleaved: bool = False, eps: float = 1e-6, positions_q=None,
                               positions_k=None, g_q_in=None, g_k_in=None, workspace=None,
                               stream=None):
    """Gradient of nt_qk_norm_rotary for the outputs' gradients g_q, g_k
    (contiguous); returns (g_q_in, g_k_in, g_w_q, g_w_k), the weights' in
    float32 (None without weights). g_q_in may be g_q and g_k_in g_k."""
    torch = _torch()
    code = _dtype_code(q)
    f32 = torch.float32
    with _On(p.device, stream) as s:
        if g_q_in is None:
            g_q_in = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k is not None and g_k_in is None:
            g_k_in = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        n = _norm_struct(p, q, k, table, interleaved, eps, g_q_in, g_k_in)
        _norm_inputs(p, n.head_dim, w_q, w_k, positions_q, positions_k)
        _flat(p, "g_q", g_q, tuple(q.shape), q.dtype)
        if k is not None:
            if g_k is None:
                raise ValueError("g_k is missing")
            _flat(p, "g_k", g_k, tuple(k.shape), q.dtype)
        g_w_q = None if w_q is None else torch.empty(n.head_dim, dtype=f32, device=q.device)
        g_w_k = None if w_k is None else torch.empty(n.head_dim, dtype=f32, device=q.device)
        need = _norm_backward_bytes(p, n, code) if w_q is not None or w_k is not None else 0
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        _expect_workspace(p, workspace, need)
        _check(_native.lib().nt_qk_norm_rotary_backward(
            ctypes.byref(p.struct), ctypes.byref(n), _at(q), _at(k), _at(g_q),
            None if k is None else _at(g_k), _at(w_q), _at(w_k), _at(table), _at(positions_q),
            _at(positions_k), _at(g_q_in), None if k is None else _at(g_k_in), _at(g_w_q),
            _at(g_w_k), code, _at(workspace), _nbytes(workspace), s))
    return g_q_in, g_k_in if k is not None else None, g_w_q, g_w_k


def _attention_struct(p, q, k, v, causal, scale):
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, head_dim]")
    heads, dim = q.shape[1], q.shape[2]
    kv = k.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(dim) if dim else 1.0
    return NtAttention(heads, kv, dim, 1 if causal else 0, scale,
                       _heads(p, "q", q, p.T, heads, dim, q.dtype),
                       _heads(p, "k", k, p.T_cols, kv, dim, q.dtype),
                       _heads(p, "v", v, p.T_cols, kv, dim, q.dtype))


def _attention_bytes(p, a, code, entry) -> int:
    b = ctypes.c_size_t()
    _check(getattr(_native.lib(), entry)(ctypes.byref(p.struct), ctypes.byref(a), code,
                                         ctypes.byref(b)))
    return b.value


def nt_attention_workspace_bytes(p: Partition, heads: int, kv_heads: int, head_dim: int,
                                 dtype, causal: bool = False) -> int:
    a = NtAttention(heads, kv_heads, head_dim, 1 if causal else 0, 1.0, 0, 0, 0)
    return _attention_bytes(p, a, _code(dtype), "nt_attention_workspace_bytes")


def nt_attention_backward_workspace_bytes(p: Partition, heads: int, kv_heads: int, head_dim: int,
                                          dtype, causal: bool = False) -> int:
    a = NtAttention(heads, kv_heads, head_dim, 1 if causal else 0, 1.0, 0, 0, 0)
    return _attention_bytes(p, a, _code(dtype), "nt_attention_backward_workspace_bytes")


def nt_single_attention(p: Partition, q, k, v, bias=None, causal: bool = False, scale=None,
                        o=None, lse=None, workspace=None, stream=None):
    """Attention of the row singles' queries q [T, heads, head_dim] over the
    column singles' keys and values [T_cols, kv_heads, head_dim] of the same
    sample, with a bias [heads, cells] from the pair state (-inf masks a
    cell) and, causal, without the keys past a query's place. scale defaults
    to 1 / sqrt(head_dim). Returns (o, lse), lse float32 [T, heads]."""
    torch = _torch()
    code = _dtype_code(q)
    with _On(p.device, stream) as s:
        a = _attention_struct(p, q, k, v, causal, scale)
        if o is None:
            o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty((p.T, a.heads), dtype=torch.float32, device=q.device)
        _flat(p, "bias", bias, (a.heads, p.cells), q.dtype)
        _flat(p, "o", o, tuple(q.shape), q.dtype)
        _flat(p, "lse", lse, (p.T, a.heads), torch.float32)
        need = _attention_bytes(p, a, code, "nt_attention_workspace_bytes")
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if workspace is not None:
            _expect_workspace(p, workspace, need)
        _check(_native.lib().nt_single_attention(
            ctypes.byref(p.struct), ctypes.byref(a), _at(q), _at(k), _at(v), _at(bias), _at(o),
            _at(lse), code, _at(workspace), 0 if workspace is None else _nbytes(workspace), s))
    return o, lse


def nt_single_attention_backward(p: Partition, q, k, v, o, lse, g_o, bias=None,
                                 causal: bool = False, scale=None, g_q=None, g_k=None, g_v=None,
                                 g_bias=None, bias_grad: bool = True, workspace=None,
                                 stream=None):
    """Gradients of nt_single_attention for g_o = dL/do (contiguous), from the
    forward's inputs, o and lse; returns (g_q, g_k, g_v, g_bias) in q's dtype
    (g_bias None without a bias, or with bias_grad False). g_q, g_k, g_v may
    be parts of one tensor, as q, k, v may."""
    torch = _torch()
    code = _dtype_code(q)
    dt = q.dtype
    with _On(p.device, stream) as s:
        a = _attention_struct(p, q, k, v, causal, scale)
        _flat(p, "bias", bias, (a.heads, p.cells), dt)
        _flat(p, "o", o, tuple(q.shape), dt)
        _flat(p, "g_o", g_o, tuple(q.shape), dt)
        _flat(p, "lse", lse, (p.T, a.heads), torch.float32)
        new = lambda t: torch.empty(t.shape, dtype=dt, device=q.device)  # noqa: E731
        g_q = new(q) if g_q is None else g_q
        g_k = new(k) if g_k is None else g_k
        g_v = new(v) if g_v is None else g_v
        if bias is None and g_bias is not None:
            raise ValueError("g_bias without a bias")
        if bias is not None and g_bias is None and bias_grad:
            g_bias = new(bias)
        _flat(p, "g_bias", g_bias, (a.heads, p.cells), dt)
        g = NtAttentionGrads(_at(g_q), _at(g_k), _at(g_v), _at(g_bias),
                             _heads(p, "g_q", g_q, p.T, a.heads, a.head_dim, dt),
                             _heads(p, "g_k", g_k, p.T_cols, a.kv_heads, a.head_dim, dt),
                             _heads(p, "g_v", g_v, p.T_cols, a.kv_heads, a.head_dim, dt))
        need = _attention_bytes(p, a, code, "nt_attention_backward_workspace_bytes")
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        _expect_workspace(p, workspace, need)
        _check(_native.lib().nt_single_attention_backward(
            ctypes.byref(p.struct), ctypes.byref(a), _at(q), _at(k), _at(v), _at(bias), _at(o),
            _at(lse), _at(g_o), ctypes.byref(g), code, _at(workspace), _nbytes(workspace), s))
    return g_q, g_k, g_v, g_bias


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
    torch = _torch()
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
    torch = _torch()
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
    torch = _torch()
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
    with _On(tensors.device, stream) as s:
        _check(_native.lib().nt_adamw_step(tensors.array, tensors.count, ctypes.byref(h),
                                           tensors.code, s))
