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
           zs=16, ws=None, n=0):
    return lib.etpc_linear(rows, n_in, n_out, dtype, x, xs, w, wi, wo, b, res, rs, act, y, ys, z, zs, ws, n, None)


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
    (dict(n_in=4096, xs=4096), WORKSPACE, "null"), (dict(n_in=4096, xs=4096, ws=E, n=64), WORKSPACE, "too small"),
    (dict(n_in=4096, xs=4096, ws=D, n=1 << 20), INVALID, "overlap"), (dict(n_in=4096, xs=4096, ws=E + 1, n=1 << 20), WORKSPACE, "aligned"),
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
    assert lib.etpc_linear_workspace_size(4, 8, 16, F32, None) == INVALID
    assert lib.etpc_linear_workspace_size(4, 8, 16, F32, C.byref(n)) == OK and n.value == 0
    assert lib.etpc_linear_backward_workspace_size(4, 8, 16, F32, 0, None) == INVALID
    assert lib.etpc_linear_backward_workspace_size(0, 8, 16, F32, 0, C.byref(n)) == OK and n.value == 0
    assert lib.etpc_linear_backward_workspace_size(1 << 30, 1 << 26, 8, F32, 0, C.byref(n)) == OVERFLOW
    assert etpc.etpc_linear_workspace_size(16, 4096, 64, torch.bfloat16) >= 16 * 64 * 4
    assert etpc.etpc_linear_workspace_size(100000, 4096, 4096, torch.bfloat16) == 0
    plain = etpc.etpc_linear_backward_workspace_size(1000, 256, 256, torch.bfloat16)
    assert etpc.etpc_linear_backward_workspace_size(1000, 256, 256, torch.bfloat16, "silu") >= plain + 1000 * 256 * 2


def test_binding_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(8, 16)
    with pytest.raises(ValueError, match="GPU"):
        etpc.etpc_linear(x, w)
    with pytest.raises(ValueError, match="act"):
        etpc.etpc_linear(x, w, act="swish")
    with pytest.raises(TypeError, match="float32"):
        etpc.etpc_linear(x.double(), w)


def join(rows=4, cols=8, dtype=F32, x=A, xs=8, gate=A + 4096, gs=8, res=A + 8192, rs=8, w1=None, b2=None, eps=1e-5, y=B, ys=8,
         h=B + 4096, hs=8, stats=B + 8192):
    return lib.etpc_norm_gate_add_norm(rows, cols, dtype, x, xs, gate, gs, res, rs, w1, None, None, None, b2, eps, y, ys, h, hs,
                                       stats, None)


@pytest.mark.parametrize("kwargs,status,word", [
    (dict(rows=-1), INVALID, "negative"), (dict(cols=0), INVALID, "column"), (dict(dtype=7), INVALID, "dtype"),
    (dict(rows=1 << 31), OVERFLOW, "n_rows"), (dict(eps=-1.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"),
    (dict(x=None), INVALID, "null x"), (dict(y=None), INVALID, "null y"), (dict(gate=A + 4097), INVALID, "aligned"),
    (dict(gs=7), INVALID, "stride"), (dict(rs=7), INVALID, "stride"), (dict(hs=7), INVALID, "stride"), (dict(ys=0), INVALID, "stride"),
    (dict(w1=D + 1), INVALID, "aligned"), (dict(stats=D + 2), INVALID, "aligned"), (dict(y=A), INVALID, "overlap"),
    (dict(h=A + 8192), INVALID, "overlap"), (dict(y=B + 4096), INVALID, "overlap"), (dict(stats=B), INVALID, "overlap"),
    (dict(w1=B), INVALID, "overlap"), (dict(b2=B + 8192), INVALID, "overlap"),
])
def test_join_refusals(kwargs, status, word):
    assert join(**kwargs) == status and word in message()


def join_backward(rows=1000, cols=8, dtype=F32, x=A, xs=8, gate=A + (1 << 16), h=A + (2 << 16), y_bar=A + (3 << 16), ys=8, h_bar=None, stats=A + (4 << 16),
                  w1=None, x_bar=B, xbs=8, gate_bar=B + (1 << 16), res_bar=B + (2 << 16), bars=(D, D + 64, D + 128, D + 192, D + 256), ws=E,
                  n=1 << 16):
    return lib.etpc_norm_gate_add_norm_backward(rows, cols, dtype, x, xs, gate, 8, h, 8, y_bar, ys, h_bar, 8, stats, w1, None, None,
                                                None, x_bar, xbs, gate_bar, 8, res_bar, 8, *bars, ws, n, None)


@pytest.mark.parametrize("kwargs,status,word", [
    (dict(rows=-1), INVALID, "negative"), (dict(cols=0), INVALID, "column"), (dict(gate=None), INVALID, "gate_bar"),
    (dict(x=None), INVALID, "null x"), (dict(h=None), INVALID, "null h"), (dict(y_bar=None), INVALID, "null y_bar"),
    (dict(stats=None), INVALID, "null stats"), (dict(xbs=7), INVALID, "stride"), (dict(ys=7), INVALID, "stride"),
    (dict(h_bar=F + 1), INVALID, "aligned"), (dict(bars=(D + 2, None, None, None, None)), INVALID, "aligned"),
    (dict(ws=None), WORKSPACE, "null"), (dict(n=8), WORKSPACE, "too small"), (dict(x_bar=A), INVALID, "overlap"),
    (dict(res_bar=B), INVALID, "overlap"), (dict(bars=(D, D, None, None, None)), INVALID, "overlap"),
    (dict(bars=(A, None, None, None, None)), INVALID, "overlap"), (dict(ws=B), INVALID, "overlap"), (dict(w1=D), INVALID, "overlap"),
])
def test_join_backward_refusals(kwargs, status, word):
    assert join_backward(**kwargs) == status and word in message()


def test_join_no_work():
    assert join(rows=0, x=None, y=None) == OK
    none = (None,) * 5
    assert join_backward(rows=0, x=None, h=None, y_bar=None, stats=None, bars=none, ws=None, n=0) == OK
    assert join_backward(x_bar=None, gate_bar=None, res_bar=None, bars=none, ws=None, n=0) == OK
    assert etpc.etpc_norm_gate_add_norm_workspace_size(0, 8) == 0
    assert etpc.etpc_norm_gate_add_norm_workspace_size(1000, 64) > 0


def clip(sizes=(8, 16), dtypes=(F32, BF16), grads=(A, B), outs=None, ord=0, max_norm=1.0, norm=D, ws=E, n=1 << 16, count=None):
    k = len(sizes)
    p = (C.c_void_p * k)(*grads)
    o = None if outs is None else (C.c_void_p * k)(*outs)
    return lib.etpc_clip_grad_norm(k if count is None else count, p, o, (C.c_int64 * k)(*sizes), (C.c_int32 * k)(*dtypes), ord,
                                   max_norm, norm, ws, n, None)


@pytest.mark.parametrize("kwargs,status,word", [
    (dict(count=-1), INVALID, "negative number"), (dict(sizes=(8, -1)), INVALID, "negative size"),
    (dict(sizes=(1 << 47, (1 << 47) + 1)), OVERFLOW, "2^48"), (dict(dtypes=(F32, 5)), INVALID, "dtype"), (dict(ord=2), INVALID, "norm"),
    (dict(norm=None), INVALID, "null norm"), (dict(norm=D + 2), INVALID, "aligned"), (dict(max_norm=-1.0), INVALID, "max_norm"),
    (dict(max_norm=float("nan")), INVALID, "max_norm"), (dict(grads=(A, None)), INVALID, "null tensor"),
    (dict(grads=(A + 2, B)), INVALID, "aligned"), (dict(outs=(A, B + 1)), INVALID, "aligned"), (dict(ws=None), WORKSPACE, "null"),
    (dict(n=8), WORKSPACE, "too small"), (dict(ws=E + 4), WORKSPACE, "doubles"), (dict(grads=(A, A)), INVALID, "overlap"),
    (dict(grads=(A, A + 16)), INVALID, "overlap"), (dict(outs=(A + 4, D + 64)), INVALID, "overlap"),
    (dict(outs=(D + 64, D + 64)), INVALID, "overlap"), (dict(outs=(B, D + 64)), INVALID, "overlap"), (dict(norm=A + 4), INVALID, "overlap"),
    (dict(ws=B), INVALID, "overlap"),
])
def test_clip_refusals(kwargs, status, word):
    assert clip(**kwargs) == status and word in message()


def test_norm_workspace():
    assert etpc.etpc_grad_norm_workspace_size([]) == 0 and etpc.etpc_grad_norm_workspace_size([0, 0]) == 0
    assert etpc.etpc_grad_norm_workspace_size([5]) == 8
    assert etpc.etpc_grad_norm_workspace_size([1] * 1000) == 8000
    assert etpc.etpc_grad_norm_workspace_size([1 << 40] * 3) == 8 * 2048


@pytest.mark.parametrize("full,empty", [(0, 3), (1, 0), (120, 1), (600, 120), (720, 120), (1080, 130), (11520, 600)])
def test_norm_scratch(full, empty):
    """What the binding allocates by the number of tensors alone is enough whichever of them are empty."""
    sizes = [0] * empty + [1 << 22] * full
    assert etpc.etpc_grad_norm_workspace_size(sizes) <= etpc._binding._norm_ws_most(full + empty)


def test_binding_lists():
    with pytest.raises(ValueError, match="ord"):
        etpc.etpc_grad_norm([torch.zeros(3)], ord=1)
    with pytest.raises(ValueError, match="GPU"):
        etpc.etpc_grad_norm([torch.zeros(3)])
