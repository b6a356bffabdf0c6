"""Host-side refusals of the operators between tokens and singles (no GPU):
every call here is invalid by construction, or has nothing to do, and launches
nothing."""
import ctypes
import math
import os

import pytest

from padding_free_pair_amd import _native as E
from test_abi_host import FAKE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(E.LIB_PATH):
        from padding_free_pair_amd import build
        build.build(verbose=False)
    return E.lib()


def at(k):
    return FAKE + 0x100000000 * (k + 1)


def embedding(lib, **change):
    a = dict(table=at(0), tokens=at(1), out=at(2), T=5, V=9, C=16, scale=1.0, dtype=1, stream=None)
    a.update(change)
    return lib.nt_token_embedding(*a.values())


def embedding_backward(lib, **change):
    a = dict(tokens=at(0), g=at(1), table=at(2), T=5000, V=9, C=16, scale=1.0, accumulate=0,
             dtype=1, ws=at(3), bytes=1 << 20, stream=None)
    a.update(change)
    return lib.nt_token_embedding_backward(*a.values())


def norm(lib, **change):
    a = dict(x=at(0), residual=at(1), w=at(2), h=at(3), y=at(4), rows=5, C=16, eps=1e-6, dtype=1,
             stream=None)
    a.update(change)
    return lib.nt_residual_norm(*a.values())


def norm_8bit(lib, **change):
    a = dict(x=at(0), residual=at(1), w=at(2), h=at(3), codes=at(4), scales=at(5), rows=5, C=384,
             group=0, eps=1e-6, dtype=1, stream=None)
    a.update(change)
    return lib.nt_residual_norm_8bit(*a.values())


def norm_backward(lib, **change):
    a = dict(h=at(0), g_y=at(1), g_h=at(2), w=at(3), g=at(4), g_w=at(5), rows=5, C=16, eps=1e-6,
             dtype=1, ws=at(6), bytes=1 << 20, stream=None)
    a.update(change)
    return lib.nt_residual_norm_backward(*a.values())


def loss(lib, **change):
    a = dict(x=at(0), W=at(1), targets=at(2), nll=at(3), lse=at(4), T=5, V=9, C=16, scale=1.0,
             dtype=1, ws=at(5), bytes=1 << 20, stream=None)
    a.update(change)
    return lib.nt_token_loss(*a.values())


def loss_backward(lib, **change):
    a = dict(x=at(0), W=at(1), targets=at(2), lse=at(3), g_nll=at(4), g_lse=at(5), g_x=at(6),
             g_W=at(7), T=5, V=9, C=16, scale=1.0, accumulate=0, dtype=1, ws=at(8),
             bytes=1 << 30, stream=None)
    a.update(change)
    return lib.nt_token_loss_backward(*a.values())


SIZES = [{"T": -1}, {"T": 2 ** 31}, {"V": 0}, {"V": -3}, {"V": 2 ** 26 + 1}, {"C": 0}, {"C": 12},
         {"C": 16392}]
ROWS = [{"rows": -1}, {"rows": 2 ** 31}, {"C": 0}, {"C": 12}, {"C": 16392}, {"eps": -1e-6},
        {"eps": math.nan}, {"eps": math.inf}]


@pytest.mark.parametrize("call,changes", [
    (embedding, SIZES + [{"scale": math.inf}, {"scale": math.nan}]),
    (embedding_backward, SIZES + [{"scale": math.nan}, {"accumulate": 2}, {"accumulate": -1}]),
    (norm, ROWS),
    (norm_8bit, ROWS + [{"group": 4}, {"group": 24}, {"group": 256}, {"group": -8}, {"group": 1024},
                        {"group": 640, "C": 640}]),
    (norm_backward, ROWS),
    (loss, SIZES + [{"scale": math.inf}, {"scale": 0.0}, {"scale": -0.0}]),
    (loss_backward, SIZES + [{"scale": math.inf}, {"scale": 0.0}, {"accumulate": 3}])])
def test_sizes(lib, call, changes):
    for change in changes:
        assert call(lib, **change) == E.NT_ERR_INVALID, change
        assert lib.nt_last_error()
    assert call(lib, dtype=7) == E.NT_ERR_DTYPE


@pytest.mark.parametrize("call", [loss, loss_backward])
def test_scales_without_a_product(lib, call):
    """Finite scales whose product with log2(e) may not be, and their neighbours."""
    for scale in (3.4e38, -3.4e38, 2.0 ** 101, math.nan, -math.inf):
        assert call(lib, scale=scale) == E.NT_ERR_INVALID, scale
    assert call(lib, scale=2.0 ** 100, bytes=0) == E.NT_ERR_WORKSPACE


@pytest.mark.parametrize("call,needed,free", [
    (embedding, ["table", "tokens", "out"], []),
    (embedding_backward, ["tokens", "g", "table", "ws"], []),
    (norm, ["x", "h", "y"], []),
    (norm_8bit, ["x", "h", "codes", "scales"], []),
    (norm_backward, ["h", "g_y", "g", "g_w", "ws"], []),
    (loss, ["x", "W", "targets", "nll", "lse", "ws"], ["targets", "nll", "lse"]),
    (loss_backward, ["x", "W", "targets", "lse", "g_nll", "ws"],
     ["targets", "lse", "g_nll", "g_lse"])])
def test_pointers(lib, call, needed, free):
    for name in needed:
        assert call(lib, **{name: None}) == E.NT_ERR_NULL, name
    if call in (embedding, embedding_backward):
        free = ["tokens"]
    for name in needed:
        wide = name not in free
        off = {name: at(20) + (8 if wide else 2)}
        assert call(lib, **off) == E.NT_ERR_ALIGN, name


@pytest.mark.parametrize("call", [embedding_backward, norm_backward, loss, loss_backward])
def test_workspace(lib, call):
    assert call(lib, bytes=0) == E.NT_ERR_WORKSPACE
    assert call(lib, bytes=255) == E.NT_ERR_WORKSPACE


@pytest.mark.parametrize("call,pairs", [
    (embedding, [("out", "table"), ("out", "tokens")]),
    (embedding_backward, [("table", "g"), ("table", "tokens"), ("ws", "g"), ("ws", "table")]),
    (norm, [("h", "w"), ("y", "w"), ("y", "h")]),
    (norm_8bit, [("codes", "w"), ("codes", "h"), ("scales", "codes"), ("scales", "x"),
                 ("codes", "x")]),
    (norm_backward, [("g", "h"), ("g", "w"), ("g_w", "g"), ("g_w", "w"), ("ws", "g"), ("ws", "h"),
                     ("ws", "g_w")]),
    (loss, [("nll", "lse"), ("nll", "x"), ("lse", "W"), ("ws", "nll"), ("ws", "targets")]),
    (loss_backward, [("g_x", "x"), ("g_W", "W"), ("g_x", "g_W"), ("ws", "g_x"), ("ws", "x"),
                     ("g_x", "lse"), ("g_W", "g_nll")])])
def test_overlaps(lib, call, pairs):
    for a, b in pairs:
        assert call(lib, **{a: at(30), b: at(30)}) == E.NT_ERR_INVALID, (a, b)
    # the same array only where it is whole
    if call is norm:
        assert call(lib, x=at(30), h=at(30) + 32) == E.NT_ERR_INVALID
        assert call(lib, residual=at(30), y=at(30) + 32) == E.NT_ERR_INVALID
        assert call(lib, x=at(30), h=at(30), y=at(30)) == E.NT_ERR_INVALID


def test_workspace_sizes(lib):
    """Bounded whatever the vocabulary: the logits' gradients come in pieces."""
    b = ctypes.c_size_t()

    def of(T, V, C, dtype=1):
        assert lib.nt_token_loss_backward_workspace_bytes(T, V, C, dtype, ctypes.byref(b)) == E.NT_OK
        return b.value

    T, C = 8192, 2048
    d = 512 << 20  # in two forms, of T x piece values each
    for V in (32003, 131072, 2 ** 20):
        # x twice, the sums of g_x, and a piece of W: as large as d at C = T
        assert of(T, V, C) <= d + T * C * (2 + 2 + 4) + d + (1 << 20)
        assert of(T, V, C, 0) <= d + T * C * (4 + 4 + 4 * 16) + d + (1 << 20)
    assert of(T, 2 ** 20, C) < T * 2 ** 20 * 2  # less than the logits would take
    # more tokens come in passes
    assert of(2 ** 24, 32003, C) == of(2 ** 16, 32003, C)
    assert of(0, 5, 8) == 0
    assert lib.nt_token_loss_backward_workspace_bytes(5, 9, 16, 1, None) == E.NT_ERR_NULL
    assert lib.nt_token_loss_workspace_bytes(5, 9, 16, 1, None) == E.NT_ERR_NULL
    assert lib.nt_token_embedding_backward_workspace_bytes(5, 9, 16, None) == E.NT_ERR_NULL
    assert lib.nt_residual_norm_backward_workspace_bytes(5, 16, None) == E.NT_ERR_NULL
    assert lib.nt_residual_norm_backward_workspace_bytes(-1, 16, ctypes.byref(b)) == E.NT_ERR_INVALID
    assert lib.nt_token_loss_workspace_bytes(5, 9, 17, 1, ctypes.byref(b)) == E.NT_ERR_INVALID
    assert lib.nt_token_loss_workspace_bytes(5, 9, 16, 9, ctypes.byref(b)) == E.NT_ERR_DTYPE


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T", [1, 16, 256, 257, 3000, 65536])
def test_workspace_of_few_tokens(lib, T, dtype):
    """No array of the loss's gradient grows with the vocabulary: neither the logits'
    gradients, of which few tokens have many rows, nor the copy of W's rows beside them."""
    b = ctypes.c_size_t()
    es, planes = (2, 2) if dtype else (4, 1)
    line, rows, mib = 128 // es, (T + 255) // 256 * 256, 1 << 20
    for C in (8, 384, 4096, 8192, 16384):
        d = max(512 * mib, 256 * (rows + line) * es * planes)
        w = max(512 * mib, (256 + line) * C * es)
        x = (2 * rows + line) * C * es
        sums = max(4 * rows * C, 256 * mib) + 256 * mib
        for V in (33, 32003, 131072, 524288, 2 ** 26):
            assert lib.nt_token_loss_backward_workspace_bytes(T, V, C, dtype,
                                                              ctypes.byref(b)) == E.NT_OK
            assert b.value <= d + w + x + sums + mib, (V, C, b.value)


def test_nothing_to_do(lib):
    """Calls without rows that write nothing return at once."""
    assert embedding(lib, T=0, tokens=None, out=None) == E.NT_OK
    assert embedding_backward(lib, T=0, tokens=None, g=None, ws=None, bytes=0,
                              accumulate=1) == E.NT_OK
    assert norm(lib, rows=0, x=None, residual=None, h=None, y=None) == E.NT_OK
    assert loss(lib, T=0, x=None, targets=None, nll=None, lse=None, ws=None, bytes=0) == E.NT_OK
    assert loss_backward(lib, T=0, x=None, targets=None, lse=None, g_nll=None, g_lse=None, g_x=None,
                         ws=None, bytes=0, accumulate=1) == E.NT_OK
