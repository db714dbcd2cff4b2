"""Refusals of operands of the node-wise operators that share memory or are not aligned, and
whole numbers as seeds (no GPU).  Every call fails its checks on the host before anything is
enqueued, so its placeholder pointers are never read."""
import ctypes as C

import numpy as np
import pytest

import equivariant_gnn_tensor_amd as etpc
from equivariant_gnn_tensor_amd import _binding

lib = etpc.lib
INVALID = 1
MB = 1 << 20
F32 = 0
ROWS, COLS = 600, 64
X, Y, H, R, M, S, W, B, WB, BB, WS = (k * MB for k in range(1, 12))
NEED = etpc.etpc_layer_norm_workspace_size(ROWS, COLS)
assert 0 < NEED < MB


def refused(status, *words):
    message = lib.etpc_last_error().decode()
    assert status == INVALID and all(w in message for w in words), (status, message)


def spec(offset_add=None):
    return C.byref(_binding.etpc_dropout_spec(0.5, 1, 2, offset_add))


def forward(y=Y, h=H, mean=M, rstd=S, w=W, b=B, offset_add=None):
    return lib.etpc_dropout_add_layer_norm(ROWS, COLS, F32, X, COLS, R, COLS, spec(offset_add), w, b, 1e-5, y, COLS, h, COLS,
                                           mean, rstd, None)


@pytest.mark.parametrize("kwargs,words", [
    (dict(mean=X + 400), ("mean", "x")), (dict(rstd=R), ("rstd", "residual")), (dict(mean=Y - 4 * ROWS + 4), ("mean", "y")),
    (dict(mean=H), ("mean", "h")), (dict(rstd=M + 4 * ROWS - 4), ("rstd", "mean")), (dict(mean=W), ("mean", "w")),
    (dict(rstd=B + 4 * COLS - 4), ("rstd", "b")), (dict(w=Y + 128), ("y", "w")), (dict(b=H), ("h", "b")),
    (dict(offset_add=Y + 256), ("y", "offset_add")), (dict(offset_add=M), ("mean", "offset_add")),
    (dict(offset_add=8 * MB + 4), ("offset_add", "aligned")), (dict(mean=M + 2), ("mean", "aligned")),
    (dict(rstd=S + 1), ("rstd", "aligned")), (dict(w=W + 2), ("w", "aligned")), (dict(b=B + 3), ("b", "aligned")),
])
def test_forward(kwargs, words):
    refused(forward(**kwargs), "overlap" if "aligned" not in words else "aligned", *words)


def backward(x_bar=Y, r_bar=R, mean=M, rstd=S, w=W, w_bar=WB, b_bar=BB, ws=WS, offset_add=None):
    return lib.etpc_dropout_add_layer_norm_backward(ROWS, COLS, F32, X, COLS, H, COLS, None, COLS, mean, rstd, w,
                                                    spec(offset_add), x_bar, COLS, r_bar, COLS, w_bar, b_bar, ws, NEED, None)


@pytest.mark.parametrize("kwargs,words", [
    (dict(w_bar=X), ("w_bar", "h")), (dict(b_bar=H), ("b_bar", "y_bar")), (dict(w_bar=Y), ("w_bar", "x_bar")),
    (dict(b_bar=R), ("b_bar", "residual_bar")), (dict(b_bar=WB + 4 * COLS - 4), ("b_bar", "w_bar")),
    (dict(w_bar=W), ("w_bar", "w")), (dict(w_bar=M), ("w_bar", "mean")), (dict(b_bar=S), ("b_bar", "rstd")),
    (dict(x_bar=M - 512), ("x_bar", "mean")), (dict(r_bar=W), ("residual_bar", "w")),
    (dict(ws=WB - NEED + 4), ("workspace", "w_bar")), (dict(ws=Y), ("workspace", "x_bar")), (dict(ws=X), ("workspace", "h")),
    (dict(ws=S), ("workspace", "rstd")), (dict(offset_add=WS + 8), ("workspace", "offset_add")),
    (dict(w_bar=WB + 2), ("w_bar", "aligned")), (dict(b_bar=BB + 1), ("b_bar", "aligned")),
    (dict(mean=M + 2), ("mean", "aligned")), (dict(rstd=S + 2), ("rstd", "aligned")), (dict(w=W + 1), ("w", "aligned")),
])
def test_backward(kwargs, words):
    refused(backward(**kwargs), "overlap" if "aligned" not in words else "aligned", *words)


def test_dropout_offset():
    refused(lib.etpc_dropout(ROWS, COLS, F32, X, COLS, spec(X + 64), X, COLS, None), "y", "offset_add", "overlap")
    refused(lib.etpc_dropout(ROWS, COLS, F32, X, COLS, spec(M + 4), Y, COLS, None), "offset_add", "aligned")
    ir = (_binding.etpc_irrep * 1)(_binding.etpc_irrep(COLS, 0, 1))
    refused(lib.etpc_irreps_dropout(1, ir, ROWS, X, spec(X + 64), X, None), "y", "offset_add", "overlap")


IR = (_binding.etpc_irrep * 2)(_binding.etpc_irrep(16, 0, 1), _binding.etpc_irrep(16, 1, -1))   # 64 numbers a row
IR_NEED = etpc.etpc_irreps_norm_workspace_size("16x0e+16x1o", ROWS)


@pytest.mark.parametrize("kwargs,words", [
    (dict(stats=X), ("stats", "x")), (dict(stats=Y - 16), ("stats", "y")), (dict(stats=W), ("stats", "w")),
    (dict(w=Y), ("y", "w")), (dict(b=Y + 4), ("y", "b")), (dict(stats=M + 2), ("stats", "aligned")),
    (dict(w=W + 1), ("w", "aligned")), (dict(b=B + 2), ("b", "aligned")),
])
def test_irreps_norm(kwargs, words):
    a = dict(w=W, b=B, stats=M) | kwargs
    st = lib.etpc_irreps_norm(2, IR, ROWS, X, a["w"], a["b"], 1e-5, Y, a["stats"], None)
    refused(st, "overlap" if "aligned" not in words else "aligned", *words)


@pytest.mark.parametrize("kwargs,words", [
    (dict(x_bar=M), ("x_bar", "stats")), (dict(x_bar=W - 16), ("x_bar", "w")), (dict(w_bar=X), ("w_bar", "x")),
    (dict(w_bar=H), ("w_bar", "y_bar")), (dict(w_bar=W), ("w_bar", "w")), (dict(b_bar=M), ("b_bar", "stats")),
    (dict(b_bar=WB + 124), ("b_bar", "w_bar")), (dict(ws=X), ("workspace", "x")), (dict(ws=WB - IR_NEED + 4), ("workspace", "w_bar")),
    (dict(w_bar=WB + 2), ("w_bar", "aligned")), (dict(b_bar=BB + 2), ("b_bar", "aligned")),
    (dict(stats=M + 2), ("stats", "aligned")),
])
def test_irreps_norm_backward(kwargs, words):
    assert 0 < IR_NEED < MB
    a = dict(stats=M, w=W, x_bar=Y, w_bar=WB, b_bar=BB, ws=WS) | kwargs
    st = lib.etpc_irreps_norm_backward(2, IR, ROWS, X, H, a["stats"], a["w"], a["x_bar"], a["w_bar"], a["b_bar"], a["ws"],
                                       IR_NEED, None)
    refused(st, "overlap" if "aligned" not in words else "aligned", *words)


@pytest.mark.parametrize("kind", [int, np.int64, np.uint64, np.int32, np.uint8])
def test_whole_numbers_as_seed_and_offset(kind):
    """Any whole number is a seed or an offset, taken modulo 2^64."""
    s = _binding._drop_spec(0.5, kind(7), kind(9), None)
    assert (s.p, s.seed, s.offset, s.offset_add) == (0.5, 7, 9, None)
    if kind not in (np.uint64, np.uint8):
        s = _binding._drop_spec(0.5, kind(-1), kind(-2), None)
        assert (s.seed, s.offset) == ((1 << 64) - 1, (1 << 64) - 2)
    for seed, offset in ((1.0, 2), (1, 2.0), ("1", 2)):
        with pytest.raises(TypeError):
            _binding._drop_spec(0.5, seed, offset, None)
