"""GPU checks of kernel paths of the node-wise operators that the sizes in
test_gpu_nodewise.py do not reach: irreps blocks taken channel by channel whose channels end
inside a vector, blocks that go channel by channel forward and flat backward, the backward
pass of 5121 to 6144 columns, and 16-bit rows of whole vectors that start at odd elements.

Oracle and tolerances are those of test_gpu_nodewise.py: a lane adds at most 56 numbers of
an irreps segment and 16 of a row before the tree, within the 256 u and 64 u counted there.
"""
import numpy as np
import pytest
import torch

from oracle import nodewise as nw
from tests.gpu_helpers import note
from tests.test_gpu_nodewise import DTYPES, EPS, U, check_backward, check_forward, close, f64, rows, tensor
from tests.test_gpu_nodewise import test_irreps_dropout as check_irreps_dropout
from tests.test_gpu_nodewise import test_irreps_norm as check_irreps_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _etpc():
    import equivariant_gnn_tensor_amd as etpc
    return etpc


# odd channel counts of 24 and more at each degree; past 256 channels; 16 to 23 channels;
# fewer than four channels beside wide ones
LISTS = ["26x1o+33x2e+45x3o", "301x1o+258x2e", "17x1o+20x2e+23x3o", "61x0e+16x3e+35x1o", "2x1o+97x3e+3x0e+131x1e", "511x1o+30x0o"]


@pytest.mark.parametrize("text", LISTS)
@pytest.mark.parametrize("n", [1, 6, 67, 2500])
def test_irreps_norm(text, n):
    check_irreps_norm(text, n)


@pytest.mark.parametrize("text", LISTS)
@pytest.mark.parametrize("n", [1, 77])
def test_irreps_dropout(text, n):
    check_irreps_dropout(text, n)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [4105, 5120, 5121, 6000, 6143, 6144, 6145])
@pytest.mark.parametrize("n", [1, 3, 600])
def test_wide_rows(kind, cols, n):
    etpc = _etpc()
    rng = np.random.default_rng(cols + n)
    note(f"layer norm {kind} rows={n} cols={cols}")
    x, yb = rows(rng, n, cols, kind), rows(rng, n, cols, kind, shift=0.0)
    w, b = tensor(rng.standard_normal(cols)), tensor(rng.standard_normal(cols))
    y, mean, rstd = etpc.etpc_layer_norm(x, w, b, eps=EPS)
    check_forward(y, mean, rstd, f64(x), np.zeros(n), f64(w), f64(b), kind)
    outs = etpc.etpc_layer_norm_backward(x, yb, mean, rstd, w)
    check_backward(*outs, f64(x), f64(yb), f64(mean), f64(rstd), f64(w), kind)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [1032, 2048, 2047, 4104, 6000, 8192, 8200])
@pytest.mark.parametrize("odd", ["h", "y_bar", "h_bar", "all"])
def test_join_backward_of_rows_from_odd_elements(kind, cols, odd):
    """Each operand in turn, then all, in rows that start at even and odd elements by turns;
    NaN around them shows any column read from a neighbour."""
    etpc = _etpc()
    rng = np.random.default_rng(cols)
    n, p, seed, off = 21, 0.25, 5, (1 << 35) + 1
    note(f"join backward {kind} cols={cols} odd={odd}")

    def operand(name, shift):
        by = 1 if odd in (name, "all") else 0
        pitch = cols + 1 + (cols + 1 + by) % 2   # odd pitch where asked for, even elsewhere
        full = torch.full((n, pitch + 2), float("nan"), dtype=DTYPES[kind], device="cuda").view(-1)
        t = full.as_strided((n, cols), (pitch, 1), by)
        t.copy_(tensor(rng.standard_normal((n, cols)) + shift, DTYPES[kind]))
        assert t.stride(0) % 2 == by and (kind == "f32" or (t.data_ptr() % 4 != 0) == bool(by))
        return t

    h, yb, hb = operand("h", 0.5), operand("y_bar", 0.0), operand("h_bar", 0.0)
    w = tensor(rng.standard_normal(cols))
    _, rm, rs = nw.layer_norm(f64(h), np.ones(cols), np.zeros(cols), EPS)
    mean, rstd = tensor(rm), tensor(rs)
    xb, rb, wb, bb = etpc.etpc_dropout_add_layer_norm_backward(h, yb, mean, rstd, w, h_bar=hb, p=p, seed=seed, offset=off)
    rx, err = check_backward(rb, wb, bb, f64(h), f64(yb), f64(mean), f64(rstd), f64(w), kind, extra=f64(hb))
    scale = 65536.0 / (65536 - nw.threshold(p))
    close(xb, nw.dropout(rx, p, seed, off), scale * (err + U * np.abs(rx)), "x_bar", kind)
    plain = etpc.etpc_layer_norm_backward(h, yb, mean, rstd, w)
    check_backward(*plain, f64(h), f64(yb), f64(mean), f64(rstd), f64(w), kind)
