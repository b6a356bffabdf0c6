"""Binding of the operators between tokens and singles: the tokens' embedding,
the singles' norm with the residual, the cross entropy over a vocabulary.

Singles are [tokens, width] tensors of all samples' tokens, contiguous, in any
partition. As in the rest of the binding, the functions check shapes and
marshal pointers, and the library computes.
"""
from __future__ import annotations

import ctypes
import functools

from . import _check, _code, _dtype_code, _native
from ._native import NT_OK
from ._single import _at, _load, _on, _workspace


def _expect(device, name, t, shape, dtype) -> None:
    """Checks a contiguous tensor (None passes)."""
    if t is None or (t.shape == shape and t.dtype == dtype and t.device == device and
                     t.is_contiguous()):
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the others on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} must be contiguous")


def _rows(name, t):
    """(rows, width) of a tensor of singles."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [tokens, width]")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, not on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.shape


def _tokens(torch, device, name, t, count) -> None:
    if t.dim() != 1:
        raise ValueError(f"{name} must be [tokens]")
    _expect(device, name, t, (count,), torch.int32)


@functools.lru_cache(maxsize=256)
def _bytes(name, *args) -> int:
    """Workspace bytes, which the sizes alone decide."""
    b = ctypes.c_size_t()
    status = getattr(_native.lib(), name)(*args, ctypes.byref(b))
    if status != NT_OK:
        _check(status)
    return b.value


def nt_token_embedding(table, tokens, scale: float = 1.0, out=None, stream=None):
    """Singles [tokens, width] of int32 tokens: scale times their rows of table
    [vocabulary, width]. Tokens below zero are absent and give zeros, tokens
    that the table does not hold NaN."""
    torch, lib = _load()
    code, dev = _dtype_code(table), table.device
    V, C = _rows("table", table)
    _tokens(torch, dev, "tokens", tokens, tokens.shape[0] if tokens.dim() else 0)
    T = tokens.shape[0]
    with _on(torch, dev, stream) as s:
        if out is None:
            out = table.new_empty((T, C))
        else:
            _expect(dev, "out", out, (T, C), table.dtype)
        status = lib.nt_token_embedding(_at(table), _at(tokens), _at(out), T, V, C, scale, code, s)
        if status != NT_OK:
            _check(status)
    return out


def nt_token_embedding_backward_workspace_bytes(tokens: int, vocabulary: int, width: int) -> int:
    return _bytes("nt_token_embedding_backward_workspace_bytes", tokens, vocabulary,
                  width)


def nt_token_embedding_backward(tokens, g_out, vocabulary: int, scale: float = 1.0, g_table=None,
                                accumulate: bool = False, workspace=None, stream=None):
    """Gradient of nt_token_embedding's table for g_out [tokens, width]: float32
    [vocabulary, width], or added to g_table with accumulate."""
    torch, lib = _load()
    code, dev = _dtype_code(g_out), g_out.device
    T, C = _rows("g_out", g_out)
    _tokens(torch, dev, "tokens", tokens, T)
    if accumulate and g_table is None:
        raise ValueError("accumulate needs g_table")
    with _on(torch, dev, stream) as s:
        need = _bytes("nt_token_embedding_backward_workspace_bytes", T, vocabulary, C)
        if g_table is None:
            g_table = torch.empty((vocabulary, C), dtype=torch.float32, device=dev)
        else:
            _expect(dev, "g_table", g_table, (vocabulary, C), torch.float32)
        ws, have, workspace = _workspace(torch, dev, workspace, need)
        status = lib.nt_token_embedding_backward(_at(tokens), _at(g_out), _at(g_table), T,
                                                 vocabulary, C, scale, 1 if accumulate else 0,
                                                 code, ws, have, s)
        if status != NT_OK:
            _check(status)
    return g_table


def _sum_of(torch, dev, x, residual, h):
    """The checked output for x + residual (x itself without a residual)."""
    if residual is None:
        if h is not None and h is not x:
            raise ValueError("h without a residual")
        return x
    _expect(dev, "residual", residual, x.shape, x.dtype)
    if h is None:
        return torch.empty_like(x)
    _expect(dev, "h", h, x.shape, x.dtype)
    return h


def nt_residual_norm(x, w=None, residual=None, eps: float = 1e-6, y=None, h=None, stream=None):
    """h = x + residual (x without one) and y = h / sqrt(mean h^2 + eps) * w over
    each row (w: float32 [width]; None: no weight); returns (y, h). h may be x or
    residual."""
    torch, lib = _load()
    code, dev = _dtype_code(x), x.device
    T, C = _rows("x", x)
    _expect(dev, "w", w, (C,), torch.float32)
    with _on(torch, dev, stream) as s:
        h = _sum_of(torch, dev, x, residual, h)
        if y is None:
            y = torch.empty_like(x)
        else:
            _expect(dev, "y", y, (T, C), x.dtype)
        status = lib.nt_residual_norm(_at(x), _at(residual), _at(w),
                                      None if residual is None else _at(h), _at(y), T, C, eps,
                                      code, s)
        if status != NT_OK:
            _check(status)
    return y, h


def nt_residual_norm_8bit(x, w=None, residual=None, eps: float = 1e-6, group: int = 0, codes=None,
                          scales=None, h=None, stream=None):
    """nt_residual_norm with y in 8 bits; returns (codes, scales, h): codes
    float8_e4m3fn [tokens, width] in units of scales, float32 [tokens, 1], or
    [tokens, width / group] with a scale for each `group` columns."""
    torch, lib = _load()
    code, dev = _dtype_code(x), x.device
    T, C = _rows("x", x)
    _expect(dev, "w", w, (C,), torch.float32)
    if group < 0 or (group and C % group):
        raise ValueError(f"group = {group} must be 0 or divide the width {C}")
    shape = (T, C // group if group else 1)
    with _on(torch, dev, stream) as s:
        h = _sum_of(torch, dev, x, residual, h)
        if codes is None:
            codes = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        else:
            _expect(dev, "codes", codes, (T, C), torch.float8_e4m3fn)
        if scales is None:
            scales = x.new_empty(shape, dtype=torch.float32)
        else:
            _expect(dev, "scales", scales, shape, torch.float32)
        status = lib.nt_residual_norm_8bit(_at(x), _at(residual), _at(w),
                                           None if residual is None else _at(h), _at(codes),
                                           _at(scales), T, C, group, eps, code, s)
        if status != NT_OK:
            _check(status)
    return codes, scales, h


def nt_residual_norm_backward_workspace_bytes(tokens: int, width: int) -> int:
    return _bytes("nt_residual_norm_backward_workspace_bytes", tokens, width)


def nt_residual_norm_backward(h, g_y, w=None, g_h=None, eps: float = 1e-6, g=None, g_w=None,
                              workspace=None, stream=None):
    """Gradient of nt_residual_norm for g_y = dL/dy and, optionally, g_h = dL/dh,
    from its h; returns (g, g_w): g for x and for the residual, g_w float32 [width]
    (None without w). g may be g_y or g_h."""
    torch, lib = _load()
    code, dev, dt = _dtype_code(h), h.device, h.dtype
    T, C = shape = _rows("h", h)
    _expect(dev, "g_y", g_y, shape, dt)
    _expect(dev, "g_h", g_h, shape, dt)
    _expect(dev, "w", w, (C,), torch.float32)
    with _on(torch, dev, stream) as s:
        if g is None:
            g = torch.empty_like(h)
        else:
            _expect(dev, "g", g, shape, dt)
        need = 0
        if w is None:
            g_w = None
        else:
            need = _bytes("nt_residual_norm_backward_workspace_bytes", T, C)
            if g_w is None:
                g_w = torch.empty_like(w)
            else:
                _expect(dev, "g_w", g_w, (C,), torch.float32)
        ws, have, workspace = _workspace(torch, dev, workspace, need)
        status = lib.nt_residual_norm_backward(_at(h), _at(g_y), _at(g_h), _at(w), _at(g),
                                               _at(g_w), T, C, eps, code, ws, have, s)
        if status != NT_OK:
            _check(status)
    return g, g_w


def nt_token_loss_workspace_bytes(tokens: int, vocabulary: int, width: int, dtype) -> int:
    return _bytes("nt_token_loss_workspace_bytes", tokens, vocabulary, width,
                  _code(dtype))


def nt_token_loss_backward_workspace_bytes(tokens: int, vocabulary: int, width: int,
                                           dtype) -> int:
    return _bytes("nt_token_loss_backward_workspace_bytes", tokens, vocabulary, width,
                  _code(dtype))


def _loss_inputs(torch, dev, x, W, targets):
    T, C = _rows("x", x)
    V = _rows("W", W)[0]
    _expect(dev, "W", W, (V, C), x.dtype)
    _tokens(torch, dev, "targets", targets, T)
    return T, V, C


def nt_token_loss(x, W, targets, scale: float = 1.0, nll=None, lse=None, workspace=None,
                  stream=None):
    """Cross entropy of singles x [tokens, width] over a vocabulary with weights
    W [vocabulary, width] for int32 targets; returns (nll, lse), float32
    [tokens], of the logits scale x W^T, which are not kept. Tokens whose target
    is below zero take no part (0 in both)."""
    torch, lib = _load()
    code, dev, f32 = _dtype_code(x), x.device, torch.float32
    T, V, C = _loss_inputs(torch, dev, x, W, targets)
    with _on(torch, dev, stream) as s:
        need = _bytes("nt_token_loss_workspace_bytes", T, V, C, code)
        if nll is None:
            nll = torch.empty((T,), dtype=f32, device=dev)
        else:
            _expect(dev, "nll", nll, (T,), f32)
        if lse is None:
            lse = torch.empty((T,), dtype=f32, device=dev)
        else:
            _expect(dev, "lse", lse, (T,), f32)
        ws, have, workspace = _workspace(torch, dev, workspace, need)
        status = lib.nt_token_loss(_at(x), _at(W), _at(targets), _at(nll), _at(lse), T, V, C,
                                   scale, code, ws, have, s)
        if status != NT_OK:
            _check(status)
    return nll, lse


def nt_token_loss_backward(x, W, targets, lse, g_nll, g_lse=None, scale: float = 1.0, g_x=None,
                           g_W=None, accumulate: bool = False, weight_grad: bool = True,
                           workspace=None, stream=None, x_grad: bool = True):
    """Gradients of nt_token_loss for g_nll = dL/dnll and, optionally, g_lse =
    dL/dlse (float32 [tokens]) from its inputs and lse; returns (g_x, g_W), g_x in
    x's dtype, g_W float32 [vocabulary, width], added to the given one with
    accumulate. With x_grad (x is nobody's output) or weight_grad (W is kept) False
    that one is None and not computed."""
    torch, lib = _load()
    code, dev, f32 = _dtype_code(x), x.device, torch.float32
    T, V, C = _loss_inputs(torch, dev, x, W, targets)
    for name, t in (("lse", lse), ("g_nll", g_nll), ("g_lse", g_lse)):
        _expect(dev, name, t, (T,), f32)
    if accumulate and g_W is None:
        raise ValueError("accumulate needs g_W")
    if g_W is not None and not weight_grad:
        raise ValueError("g_W without weight_grad")
    if g_x is not None and not x_grad:
        raise ValueError("g_x without x_grad")
    if not (x_grad or weight_grad):
        raise ValueError("neither x_grad nor weight_grad: nothing to compute")
    with _on(torch, dev, stream) as s:
        need = _bytes("nt_token_loss_backward_workspace_bytes", T, V, C, code)
        if g_x is not None:
            _expect(dev, "g_x", g_x, (T, C), x.dtype)
        elif x_grad:
            g_x = torch.empty_like(x)
        if g_W is not None:
            _expect(dev, "g_W", g_W, (V, C), f32)
        elif weight_grad:
            g_W = torch.empty((V, C), dtype=f32, device=dev)
        ws, have, workspace = _workspace(torch, dev, workspace, need)
        status = lib.nt_token_loss_backward(_at(x), _at(W), _at(targets), _at(lse), _at(g_nll),
                                            _at(g_lse), _at(g_x), _at(g_W), T, V, C, scale,
                                            1 if accumulate else 0, code, ws, have, s)
        if status != NT_OK:
            _check(status)
    return g_x, g_W
