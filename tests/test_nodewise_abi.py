"""Refusals of the node-wise operators (no GPU): every call below fails its checks on the host
before anything is enqueued, so its placeholder pointers are never read."""
import ctypes as C

import pytest
import torch

import equivariant_gnn_tensor_amd as etpc
from equivariant_gnn_tensor_amd import _binding

OK, INVALID, UNSUPPORTED, WORKSPACE, OVERFLOW = 0, 1, 2, 4, 5
A, B, D, E = 1 << 20, 2 << 20, 3 << 20, 4 << 20   # placeholder addresses, far apart
F32, BF16 = 0, 1
lib = etpc.lib


def message():
    return etpc.lib.etpc_last_error().decode()


def drop(p=0.5):
    return C.byref(_binding.etpc_dropout_spec(p, 1, 2, None))


def irreps(*blocks):
    return len(blocks), (_binding.etpc_irrep * max(1, len(blocks)))(*[_binding.etpc_irrep(*b) for b in blocks])


def norm(rows=4, cols=8, dtype=F32, x=A, xs=8, eps=1e-5, y=B, ys=8):
    return lib.etpc_layer_norm(rows, cols, dtype, x, xs, None, None, eps, y, ys, None, None, None)


@pytest.mark.parametrize("kwargs,status,word", [
    (dict(rows=-1), INVALID, "negative"), (dict(cols=-1), INVALID, "negative"), (dict(cols=0), INVALID, "column"),
    (dict(dtype=3), INVALID, "dtype"), (dict(dtype=-1), INVALID, "dtype"),
    (dict(rows=1 << 31), OVERFLOW, "n_rows"), (dict(cols=(1 << 30) + 1), OVERFLOW, "n_cols"),
    (dict(x=None), INVALID, "null x"), (dict(y=None), INVALID, "null y"),
    (dict(x=A + 2), INVALID, "aligned"), (dict(y=B + 1, dtype=BF16), INVALID, "aligned"),
    (dict(xs=7), INVALID, "stride"), (dict(ys=0), INVALID, "stride"), (dict(xs=-8), INVALID, "stride"),
    (dict(xs=1 << 60), OVERFLOW, "stride"),
    (dict(eps=-1.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"), (dict(eps=float("inf")), INVALID, "eps"),
    (dict(y=A), INVALID, "overlap"), (dict(y=A + 4), INVALID, "overlap"), (dict(xs=16, ys=16, y=A + 28), INVALID, "overlap"),
    (dict(xs=16, ys=24, y=A + 32), INVALID, "overlap"),
])
def test_layer_norm_refusals(kwargs, status, word):
    assert norm(**kwargs) == status and word in message()


def test_no_rows_is_no_work():
    assert norm(rows=0, x=None, y=None) == OK
    assert lib.etpc_dropout(0, 8, F32, None, 8, drop(), None, 8, None) == OK
    assert lib.etpc_dropout(8, 0, F32, None, 8, drop(), None, 8, None) == OK
    n, ir = irreps((8, 0, 1))
    assert lib.etpc_irreps_norm(n, ir, 0, None, None, None, 1e-5, None, None, None) == OK
    assert lib.etpc_irreps_dropout(n, ir, 0, None, drop(), None, None) == OK
    assert lib.etpc_irreps_norm(0, None, 5, A, None, None, 1e-5, B, None, None) == OK


@pytest.mark.parametrize("p", [-0.1, 1.5, float("nan"), float("inf")])
def test_dropout_probability(p):
    assert lib.etpc_dropout(4, 8, F32, A, 8, drop(p), B, 8, None) == INVALID and "probability" in message()
    st = lib.etpc_dropout_add_layer_norm(4, 8, F32, A, 8, None, 0, drop(p), None, None, 1e-5, B, 8, None, 0, None, None,
                                         None)
    assert st == INVALID and "probability" in message()
    n, ir = irreps((8, 0, 1))
    assert lib.etpc_irreps_dropout(n, ir, 4, A, drop(p), B, None) == INVALID


def test_dropout_refusals():
    assert lib.etpc_dropout(4, 8, F32, A, 8, None, B, 8, None) == INVALID and "spec" in message()
    assert lib.etpc_dropout(4, 8, F32, A, 8, drop(), A + 4, 8, None) == INVALID and "overlap" in message()
    assert lib.etpc_dropout(4, 8, F32, A, 8, drop(), A, 16, None) == INVALID and "overlap" in message()   # not in place
    assert lib.etpc_dropout(4, 8, F32, A, 0, drop(), A, 8, None) == INVALID
    assert lib.etpc_dropout(4, 8, 7, A, 8, drop(), B, 8, None) == INVALID and "dtype" in message()


def backward(rows=4, cols=8, h=A, yb=B, hb=None, mean=D, rstd=D, x_bar=E, r_bar=None, w_bar=None, ws=None, ws_bytes=0):
    return lib.etpc_dropout_add_layer_norm_backward(rows, cols, F32, h, cols, yb, cols, hb, cols, mean, rstd, None, None,
                                                    x_bar, cols, r_bar, cols, w_bar, None, ws, ws_bytes, None)


@pytest.mark.parametrize("kwargs,status,word", [
    (dict(h=None), INVALID, "null h"), (dict(yb=None), INVALID, "null y_bar"), (dict(mean=None), INVALID, "mean"),
    (dict(rstd=None), INVALID, "rstd"), (dict(x_bar=A), INVALID, "overlap"), (dict(r_bar=B), INVALID, "overlap"),
    (dict(r_bar=E), INVALID, "overlap"), (dict(hb=E), INVALID, "overlap"), (dict(hb=A + 2), INVALID, "aligned"),
    (dict(rows=5000, cols=64, h=1 << 30, yb=1 << 31, x_bar=1 << 32, w_bar=D), WORKSPACE, "workspace"),
    (dict(rows=5000, cols=64, h=1 << 30, yb=1 << 31, x_bar=1 << 32, w_bar=D, ws=E, ws_bytes=64), WORKSPACE, "small"),
    (dict(rows=5000, cols=64, h=1 << 30, yb=1 << 31, x_bar=1 << 32, w_bar=D, ws=E + 2, ws_bytes=1 << 40), WORKSPACE, "aligned"),
    (dict(cols=0), INVALID, "column"),
])
def test_backward_refusals(kwargs, status, word):
    assert backward(**kwargs) == status and word in message()


def test_nothing_asked_is_no_work():
    assert backward(x_bar=None) == OK


def test_workspace_sizes():
    """Partial sums of the parameter gradients: none for one workgroup, never more than
    1024 rows of them, whatever the number of rows."""
    assert etpc.etpc_layer_norm_workspace_size(1, 512) == 0
    assert etpc.etpc_layer_norm_workspace_size(0, 512) == 0 and etpc.etpc_layer_norm_workspace_size(5, 0) == 0
    for cols in (1, 64, 1000, 4096, 20000):
        for rows in (1, 5, 1000, 1 << 20, (1 << 31) - 1):
            assert etpc.etpc_layer_norm_workspace_size(rows, cols) <= 1024 * 2 * cols * 4
    assert etpc.etpc_irreps_norm_workspace_size("8x0e+8x1o", 1) == 0
    assert 0 < etpc.etpc_irreps_norm_workspace_size("8x0e+8x1o", (1 << 31) - 1) <= 1024 * 24 * 4
    with pytest.raises(etpc.EtpcError):
        etpc.etpc_layer_norm_workspace_size(-1, 8)
    with pytest.raises(etpc.EtpcError):
        etpc.etpc_irreps_norm_workspace_size("8x0e", -1)


@pytest.mark.parametrize("blocks,status", [
    ([(0, 0, 1)], INVALID), ([(-3, 0, 1)], INVALID), ([(4, 4, 1)], UNSUPPORTED), ([(4, -1, 1)], INVALID),
    ([(4, 1, 0)], INVALID), ([(4, 1, 2)], INVALID), ([(1, 0, 1)] * 65, UNSUPPORTED), ([(1 << 30, 1, 1)], OVERFLOW),
])
def test_irreps_refusals(blocks, status):
    n, ir = irreps(*blocks)
    assert lib.etpc_irreps_dims(n, ir, None, None, None) == status
    assert lib.etpc_irreps_norm(n, ir, 4, A, None, None, 1e-5, B, None, None) == status
    assert lib.etpc_irreps_dropout(n, ir, 4, A, drop(), B, None) == status


def test_irreps_norm_refusals():
    n, ir = irreps((4, 0, 1), (2, 1, -1))
    assert lib.etpc_irreps_dims(2, None, None, None, None) == INVALID
    assert lib.etpc_irreps_norm(n, ir, -1, A, None, None, 1e-5, B, None, None) == INVALID
    assert lib.etpc_irreps_norm(n, ir, 4, A, None, None, -1e-5, B, None, None) == INVALID and "eps" in message()
    assert lib.etpc_irreps_norm(n, ir, 4, A, None, None, 1e-5, A, None, None) == INVALID and "overlap" in message()
    assert lib.etpc_irreps_norm(n, ir, 4, A + 1, None, None, 1e-5, B, None, None) == INVALID
    assert lib.etpc_irreps_norm_backward(n, ir, 4, A, B, None, None, E, None, None, None, 0, None) == INVALID
    assert "stats" in message()
    assert lib.etpc_irreps_norm_backward(n, ir, 4000, A, 1 << 30, D, None, None, E, None, None, 0, None) == WORKSPACE
    assert lib.etpc_irreps_dropout(n, ir, 4, A, None, B, None) == INVALID and "spec" in message()
    assert etpc.etpc_irreps_dims("4x0e+2x1o+3x0o") == dict(dim=13, channels=9, biases=4)


def test_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        etpc.etpc_layer_norm(x)
    with pytest.raises(ValueError, match="GPU"):
        etpc.etpc_dropout(x, 0.1, 0)
    with pytest.raises(TypeError, match="float32"):
        etpc.etpc_layer_norm(x.double())
    with pytest.raises(ValueError, match="shape"):
        etpc.etpc_irreps_norm("4x0e", x)
    with pytest.raises(ValueError, match="irrep"):
        etpc.etpc_irreps_norm("4y0e", x)
