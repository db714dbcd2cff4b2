"""Refusals of the feed-forward operators (no GPU): every call below fails its checks on the
host before anything is enqueued, so its placeholder pointers are never read."""
import ctypes as C

import pytest
import torch

import equivariant_gnn_tensor_amd as etpc

OK, INVALID, UNSUPPORTED, WORKSPACE, OVERFLOW = 0, 1, 2, 4, 5
A, B, D, E, F = 1 << 24, 2 << 24, 3 << 24, 4 << 24, 5 << 24   # placeholder addresses, far apart
F32, BF16 = 0, 1
SILU = 2
lib = etpc.lib


def message():
    return etpc.lib.etpc_last_error().decode()


def linear(rows=4, n_in=8, n_out=16, dtype=F32, x=A, xs=8, w=B, wi=16, wo=1, b=None, res=None, rs=16, act=0, y=D, ys=16, z=None,
           zs=16):
    return lib.etpc_linear(rows, n_in, n_out, dtype, x, xs, w, wi, wo, b, res, rs, act, y, ys, z, zs, None)


@pytest.mark.parametrize("kwargs,status,word", [
    (dict(rows=-1), INVALID, "negative"), (dict(n_in=-1), INVALID, "at least one"), (dict(n_in=0), INVALID, "at least one"),
    (dict(n_out=0), INVALID, "at least one"), (dict(dtype=3), INVALID, "dtype"), (dict(act=5), INVALID, "activation"),
    (dict(act=-1), INVALID, "activation"),
    (dict(rows=1 << 31), OVERFLOW, "n_rows"), (dict(n_in=(1 << 30) + 1), OVERFLOW, "n_cols"),
    (dict(n_out=(1 << 30) + 1), OVERFLOW, "n_cols"), (dict(rows=1 << 30, n_in=1 << 30), OVERFLOW, "2^56"),
    (dict(n_in=1 << 29, n_out=1 << 29), OVERFLOW, "2^56"),
    (dict(x=None), INVALID, "null x"), (dict(w=None), INVALID, "null w"), (dict(y=None), INVALID, "null y"),
    (dict(x=A + 2), INVALID, "aligned"), (dict(w=B + 1, dtype=BF16), INVALID, "aligned"), (dict(b=E + 2), INVALID, "aligned"),
    (dict(xs=7), INVALID, "stride"), (dict(ys=15), INVALID, "stride"), (dict(ys=0), INVALID, "stride"),
    (dict(wi=15), INVALID, "stride"), (dict(wi=2, wo=2), INVALID, "strides must be 1"), (dict(wi=1, wo=7), INVALID, "stride"),
    (dict(res=E, rs=15), INVALID, "stride"), (dict(z=E, zs=15), INVALID, "stride"), (dict(xs=1 << 60), OVERFLOW, "stride"),
    (dict(y=A), INVALID, "overlap"), (dict(y=B + 8), INVALID, "overlap"), (dict(res=D), INVALID, "overlap"),
    (dict(z=D + 32), INVALID, "overlap"), (dict(b=D), INVALID, "overlap"),
])
def test_linear_refusals(kwargs, status, word):
    assert linear(**kwargs) == status and word in message()


def backward(rows=4, n_in=8, n_out=16, dtype=F32, x=A, xs=8, w=B, wi=16, wo=1, y_bar=D, ys=16, z=E, zs=16, act=SILU, x_bar=F,
             xbs=8, w_bar=F + 4096, wbi=16, wbo=1, b_bar=F + 8192, ws=F + 65536, n=1 << 20):
    return lib.etpc_linear_backward(rows, n_in, n_out, dtype, x, xs, w, wi, wo, y_bar, ys, z, zs, act, x_bar, xbs, w_bar, wbi,
                                    wbo, b_bar, ws, n, None)


@pytest.mark.parametrize("kwargs,status,word", [
    (dict(rows=-1), INVALID, "negative"), (dict(n_out=0), INVALID, "at least one"), (dict(act=9), INVALID, "activation"),
    (dict(x=None), INVALID, "null x"), (dict(w=None), INVALID, "null w"), (dict(y_bar=None), INVALID, "null y_bar"),
    (dict(z=None), INVALID, "null z"), (dict(xs=7), INVALID, "stride"), (dict(xbs=7), INVALID, "stride"),
    (dict(wbi=15), INVALID, "stride"), (dict(wbi=0), INVALID, "stride"), (dict(wbi=3, wbo=3), INVALID, "strides must be 1"),
    (dict(ys=15), INVALID, "stride"), (dict(b_bar=F + 8194), INVALID, "aligned"), (dict(ws=None), WORKSPACE, "null"),
    (dict(n=16), WORKSPACE, "too small"), (dict(ws=F + 65538), WORKSPACE, "aligned"), (dict(x_bar=A), INVALID, "overlap"),
    (dict(w_bar=B), INVALID, "overlap"), (dict(b_bar=F), INVALID, "overlap"), (dict(ws=D), INVALID, "overlap"),
    (dict(w_bar=F + 64), INVALID, "overlap"), (dict(x_bar=E), INVALID, "overlap"),
])
def test_linear_backward_refusals(kwargs, status, word):
    assert backward(**kwargs) == status and word in message()


def test_no_rows_is_no_work():
    assert linear(rows=0, x=None, w=None, y=None) == OK
    assert backward(rows=0, x=None, y_bar=None, z=None, w_bar=None, b_bar=None, ws=None, n=0) == OK
    assert backward(x=None, w=None, x_bar=None, w_bar=None, b_bar=None, ws=None, n=0) == OK


def test_linear_workspace():
    n = C.c_size_t()
    assert lib.etpc_linear_workspace_size(4, 8, 16, F32, 0, None) == INVALID
    assert lib.etpc_linear_workspace_size(0, 8, 16, F32, 0, C.byref(n)) == OK and n.value == 0
    assert lib.etpc_linear_workspace_size(1 << 30, 1 << 26, 8, F32, 0, C.byref(n)) == OVERFLOW
    assert etpc.etpc_linear_workspace_size(1000, 64, 64, torch.bfloat16, "silu") >= 1000 * 64 * 2
    assert etpc.etpc_linear_workspace_size(1000, 64, 64, torch.bfloat16) < 1000 * 64 * 2


def test_binding_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(8, 16)
    with pytest.raises(ValueError, match="GPU"):
        etpc.etpc_linear(x, w)
    with pytest.raises(ValueError, match="act"):
        etpc.etpc_linear(x, w, act="swish")
    with pytest.raises(TypeError, match="float32"):
        etpc.etpc_linear(x.double(), w)
