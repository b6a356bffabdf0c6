"""Host-side refusals of the single attention operators and of the AdamW step
(no GPU): every call here is invalid by construction and launches nothing."""
import ctypes
import math
import os

import pytest

from padding_free_pair_amd import _native as E
from test_abi_host import FAKE, fake_partition


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(E.LIB_PATH):
        from padding_free_pair_amd import build
        build.build(verbose=False)
    return E.lib()


def at(k):
    return FAKE + 0x10000000 * (k + 1)


def test_struct_layouts():
    assert ctypes.sizeof(E.NtRotary) == 8 + 6 * 8
    assert ctypes.sizeof(E.NtNormRotary) == 24 + 5 * 8 and E.NtNormRotary.positions.offset == 24
    assert ctypes.sizeof(E.NtAttention) == 24 + 3 * 8 and E.NtAttention.ld_q.offset == 24
    assert ctypes.sizeof(E.NtAttentionGrads) == 7 * 8
    assert ctypes.sizeof(E.NtAdamwTensor) == 8 * 8
    assert ctypes.sizeof(E.NtAdamw) == 9 * 8


@pytest.mark.parametrize("change,status", [
    ({"rot_dim": 0}, E.NT_ERR_INVALID), ({"rot_dim": 7}, E.NT_ERR_INVALID),
    ({"rot_dim": 130}, E.NT_ERR_INVALID), ({"base": 1.0}, E.NT_ERR_INVALID),
    ({"base": math.inf}, E.NT_ERR_INVALID), ({"scaling": 3}, E.NT_ERR_INVALID),
    ({"scaling": 1, "factor": 0.5}, E.NT_ERR_INVALID),
    ({"scaling": 2, "original": 0.0}, E.NT_ERR_INVALID),
    ({"scaling": 2, "beta_fast": 1.0}, E.NT_ERR_INVALID),
    ({"scaling": 2, "beta_slow": -1.0}, E.NT_ERR_INVALID),
    ({"magnitude": 0.0}, E.NT_ERR_INVALID), ({"magnitude": math.nan}, E.NT_ERR_INVALID)])
def test_rotary_table_refuses(lib, change, status):
    v = dict(rot_dim=8, scaling=0, base=1e4, factor=2.0, original=64.0, beta_fast=32.0,
             beta_slow=1.0, magnitude=1.0)
    v.update(change)
    r = E.NtRotary(*[v[k] for k in ("rot_dim", "scaling", "base", "factor", "original",
                                    "beta_fast", "beta_slow", "magnitude")])
    assert lib.nt_rotary_table(ctypes.byref(r), at(0), 4, None) == status
    assert lib.nt_last_error()


def test_rotary_table_arguments(lib):
    r = E.NtRotary(8, 0, 1e4, 1.0, 0.0, 32.0, 1.0, 1.0)
    assert lib.nt_rotary_table(None, at(0), 4, None) == E.NT_ERR_NULL
    assert lib.nt_rotary_table(ctypes.byref(r), None, 4, None) == E.NT_ERR_NULL
    assert lib.nt_rotary_table(ctypes.byref(r), at(0) + 4, 4, None) == E.NT_ERR_ALIGN
    assert lib.nt_rotary_table(ctypes.byref(r), at(0), -1, None) == E.NT_ERR_INVALID
    assert lib.nt_rotary_table(ctypes.byref(r), None, 0, None) == E.NT_OK  # nothing to write


def norm(**change):
    v = dict(heads=4, kv_heads=2, head_dim=16, rot_dim=16, interleaved=0, eps=1e-6, positions=8,
             ld_q=0, ld_k=0, ld_q_out=0, ld_k_out=0)
    v.update(change)
    return E.NtNormRotary(*v.values())


def call_norm(lib, n, p=None, ptrs=None, dtype=1, **named):
    a = dict(q=at(0), k=at(1), w_q=at(2), w_k=at(3), table=at(4), pos_q=None, pos_k=None,
             q_out=at(5), k_out=at(6))
    a.update(named)
    p = p or fake_partition()
    return lib.nt_qk_norm_rotary(ctypes.byref(p), ctypes.byref(n), *a.values(), dtype, None)


@pytest.mark.parametrize("change", [
    {"heads": 0}, {"heads": 20000}, {"kv_heads": -1}, {"head_dim": 12}, {"head_dim": 136},
    {"rot_dim": 18}, {"rot_dim": 5}, {"rot_dim": -2}, {"interleaved": 2}, {"eps": -1.0},
    {"eps": math.nan}, {"positions": 0}, {"ld_q": 56}, {"ld_q": 68}, {"ld_k": 24},
    {"ld_q_out": 60}, {"ld_q": 1 << 40}])
def test_norm_refuses(lib, change):
    assert call_norm(lib, norm(**change)) == E.NT_ERR_INVALID, change


def test_norm_arguments(lib):
    n = norm()
    raw = E.NtPartition()
    assert call_norm(lib, n, p=raw) == E.NT_ERR_INVALID
    assert call_norm(lib, n, dtype=5) == E.NT_ERR_DTYPE
    for name in ("q", "k", "table", "q_out", "k_out"):
        assert call_norm(lib, n, **{name: None}) == E.NT_ERR_NULL, name
    for k, name in enumerate(("q", "k", "w_q", "w_k", "table")):
        assert call_norm(lib, n, **{name: at(k) + 8}) == E.NT_ERR_ALIGN, name
    assert call_norm(lib, n, pos_q=at(7) + 4) == E.NT_ERR_ALIGN
    # outputs that meet an input in part, or one another
    assert call_norm(lib, n, q_out=at(0) + 32) == E.NT_ERR_INVALID
    assert call_norm(lib, n, q_out=at(1)) == E.NT_ERR_INVALID
    assert call_norm(lib, n, k_out=at(5)) == E.NT_ERR_INVALID
    assert call_norm(lib, n, q_out=at(4)) == E.NT_ERR_INVALID
    assert call_norm(lib, n, k_out=at(3) - 16) == E.NT_ERR_INVALID
    # in one fused array: the same ld, columns that meet
    f = norm(ld_q=128, ld_k=128, ld_q_out=128, ld_k_out=128)
    assert call_norm(lib, f, k=at(0) + 128, q_out=at(0) + 96, k_out=at(0) + 192) == E.NT_ERR_INVALID


def test_norm_backward_arguments(lib):
    p, n = fake_partition(), norm()
    need = ctypes.c_size_t()
    args = [ctypes.byref(p), ctypes.byref(n), 1]
    assert lib.nt_qk_norm_rotary_backward_workspace_bytes(*args, None) == E.NT_ERR_NULL
    assert lib.nt_qk_norm_rotary_backward_workspace_bytes(*args, ctypes.byref(need)) == E.NT_OK
    assert need.value > 0

    def call(have=need.value, **named):
        a = dict(q=at(0), k=at(1), g_q=at(2), g_k=at(3), w_q=at(4), w_k=at(5), table=at(6),
                 pos_q=None, pos_k=None, gi_q=at(7), gi_k=at(8), gw_q=at(9), gw_k=at(10))
        ws = named.pop("ws", at(11))
        a.update(named)
        return lib.nt_qk_norm_rotary_backward(ctypes.byref(p), ctypes.byref(n), *a.values(), 1,
                                              ws, have, None)

    assert call(have=need.value - 1) == E.NT_ERR_WORKSPACE
    assert call(ws=None) == E.NT_ERR_NULL
    assert call(ws=at(11) + 8) == E.NT_ERR_ALIGN
    for name in ("q", "g_q", "g_k", "gi_q", "gi_k", "gw_q", "gw_k"):
        assert call(**{name: None}) == E.NT_ERR_NULL, name
    assert call(gi_q=at(0)) == E.NT_ERR_INVALID   # q is read again by the weights' sums
    assert call(gi_q=at(3)) == E.NT_ERR_INVALID
    assert call(gw_q=at(10)) == E.NT_ERR_INVALID
    assert call(gw_k=at(11)) == E.NT_ERR_INVALID
    assert call(ws=at(0)) == E.NT_ERR_INVALID


def attention(**change):
    v = dict(heads=4, kv_heads=2, head_dim=16, causal=0, scale=0.25, ld_q=0, ld_k=0, ld_v=0)
    v.update(change)
    return E.NtAttention(*v.values())


BAD_ATTENTION = [{"heads": 0}, {"heads": 3}, {"kv_heads": 0}, {"kv_heads": 3}, {"head_dim": 0},
                 {"head_dim": 20}, {"head_dim": 256}, {"causal": 2}, {"scale": math.inf},
                 {"scale": math.nan}, {"ld_q": 32}, {"ld_k": 36}, {"ld_v": 1 << 40}]


def call_attention(lib, a, p=None, dtype=1, have=1 << 24, ws=at(9), **named):
    x = dict(q=at(0), k=at(1), v=at(2), bias=None, o=at(4), lse=at(5))
    x.update(named)
    p = p or fake_partition()
    return lib.nt_single_attention(ctypes.byref(p), ctypes.byref(a), *x.values(), dtype, ws, have,
                                   None)


def call_backward(lib, a, p=None, dtype=1, have=1 << 24, ws=at(20), grads=None, **named):
    x = dict(q=at(0), k=at(1), v=at(2), bias=at(3), o=at(4), lse=at(5), g_o=at(6))
    x.update(named)
    g = dict(q=at(7), k=at(8), v=at(9), bias=at(10), ld_q=0, ld_k=0, ld_v=0)
    g.update(grads or {})
    p = p or fake_partition()
    return lib.nt_single_attention_backward(ctypes.byref(p), ctypes.byref(a), *x.values(),
                                            ctypes.byref(E.NtAttentionGrads(*g.values())), dtype,
                                            ws, have, None)


@pytest.mark.parametrize("change", BAD_ATTENTION)
def test_attention_refuses(lib, change):
    assert call_attention(lib, attention(**change)) == E.NT_ERR_INVALID, change
    assert call_backward(lib, attention(**change)) == E.NT_ERR_INVALID, change


def test_attention_arguments(lib):
    a, p = attention(), fake_partition()
    n = ctypes.c_size_t()
    for entry in (lib.nt_attention_workspace_bytes, lib.nt_attention_backward_workspace_bytes):
        assert entry(ctypes.byref(p), ctypes.byref(a), 1, ctypes.byref(n)) == E.NT_OK
        assert entry(ctypes.byref(p), ctypes.byref(a), 1, None) == E.NT_ERR_NULL
        assert entry(ctypes.byref(p), None, 1, ctypes.byref(n)) == E.NT_ERR_NULL
        assert entry(ctypes.byref(p), ctypes.byref(a), 9, ctypes.byref(n)) == E.NT_ERR_DTYPE
    assert call_attention(lib, a, p=E.NtPartition()) == E.NT_ERR_INVALID
    assert call_attention(lib, a, dtype=2) == E.NT_ERR_DTYPE
    for name in ("q", "k", "v", "o", "lse"):
        assert call_attention(lib, a, **{name: None}) == E.NT_ERR_NULL, name
        assert call_attention(lib, a, **{name: at(15) + 4}) == E.NT_ERR_ALIGN, name
    assert call_attention(lib, a, bias=at(3) + 2) == E.NT_ERR_ALIGN
    for name in ("q", "k", "v"):
        assert call_attention(lib, a, **{name: at(4) + 16}) == E.NT_ERR_INVALID, name
    assert call_attention(lib, a, bias=at(4) - 16) == E.NT_ERR_INVALID
    assert call_attention(lib, a, lse=at(4)) == E.NT_ERR_INVALID


def test_attention_backward_arguments(lib):
    a, p = attention(), fake_partition()
    n = ctypes.c_size_t()
    assert lib.nt_attention_backward_workspace_bytes(ctypes.byref(p), ctypes.byref(a), 1,
                                                     ctypes.byref(n)) == E.NT_OK
    if n.value:
        assert call_backward(lib, a, have=n.value - 1) == E.NT_ERR_WORKSPACE
        assert call_backward(lib, a, ws=None) == E.NT_ERR_NULL
        assert call_backward(lib, a, ws=at(7)) == E.NT_ERR_INVALID
    for name in ("q", "k", "v", "o", "lse", "g_o"):
        assert call_backward(lib, a, **{name: None}) == E.NT_ERR_NULL, name
    for name in ("q", "k", "v"):
        assert call_backward(lib, a, grads={name: None}) == E.NT_ERR_NULL, name
        assert call_backward(lib, a, grads={name: at(0)}) == E.NT_ERR_INVALID, name
        assert call_backward(lib, a, grads={"ld_" + name: 20}) == E.NT_ERR_INVALID, name
    assert call_backward(lib, a, grads={"k": at(9)}) == E.NT_ERR_INVALID
    assert call_backward(lib, a, grads={"bias": at(3)}) == E.NT_ERR_INVALID
    assert call_backward(lib, a, grads={"q": at(5)}) == E.NT_ERR_INVALID


def tensor(k=0, **change):
    v = dict(param=at(k), grad=at(k + 1), master=None, m=at(k + 2), v=at(k + 3), m_scale=None,
             v_scale=None, n=100)
    v.update(change)
    return E.NtAdamwTensor(*v.values())


def call_adamw(lib, *tensors, dtype=0, count=None, **change):
    v = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=1, step_device=None,
             lr_device=None, state_bits=32)
    v.update(change)
    arr = (E.NtAdamwTensor * max(1, len(tensors)))(*tensors)
    h = E.NtAdamw(*v.values())
    return lib.nt_adamw_step(arr, len(tensors) if count is None else count, ctypes.byref(h), dtype,
                             None)


@pytest.mark.parametrize("change", [
    {"beta1": 1.0}, {"beta1": -0.1}, {"beta2": 1.0}, {"beta2": math.nan}, {"eps": -1.0},
    {"lr": math.inf}, {"weight_decay": math.nan}, {"step": 0}, {"state_bits": 16}, {"count": -1}])
def test_adamw_refuses(lib, change):
    assert call_adamw(lib, tensor(), **change) == E.NT_ERR_INVALID, change


def test_adamw_arguments(lib):
    assert lib.nt_adamw_step(None, 1, None, 0, None) == E.NT_ERR_NULL
    assert call_adamw(lib, dtype=3) == E.NT_ERR_DTYPE
    assert call_adamw(lib) == E.NT_OK  # no tensors: nothing to do
    for name in ("param", "grad", "m", "v"):
        assert call_adamw(lib, tensor(**{name: None})) == E.NT_ERR_NULL, name
        assert call_adamw(lib, tensor(**{name: at(9) + 4})) == E.NT_ERR_ALIGN, name
    assert call_adamw(lib, tensor(), state_bits=8) == E.NT_ERR_NULL  # no scales
    assert call_adamw(lib, tensor(n=-1)) == E.NT_ERR_INVALID
    assert call_adamw(lib, tensor(n=1 << 40)) == E.NT_ERR_INVALID
    assert call_adamw(lib, tensor(), tensor()) == E.NT_ERR_INVALID            # listed twice
    assert call_adamw(lib, tensor(), tensor(4, grad=at(2))) == E.NT_ERR_INVALID  # m as a gradient
    assert call_adamw(lib, tensor(), tensor(4, m=at(0) + 384)) == E.NT_ERR_INVALID
    assert call_adamw(lib, tensor(master=at(0))) == E.NT_ERR_INVALID
    assert call_adamw(lib, tensor(), step_device=at(0) + 8) == E.NT_ERR_INVALID
    assert call_adamw(lib, tensor(), step_device=at(9) + 4) == E.NT_ERR_ALIGN
    assert call_adamw(lib, tensor(n=0, param=None, grad=None, m=None, v=None)) == E.NT_OK
