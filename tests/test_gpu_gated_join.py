"""GPU checks of the gated join between two norms against oracle/feedforward.py (float64).

Tolerances: those of the layer norm (tests/test_gpu_nodewise.py: sums of a row 64 u, sums over rows
512 u of their terms' magnitudes, u = 2^-24), carried through the formulas.  The logistic function is
off by its exp (2 u times 2 + |gate| to first order) and a few roundings, counted as
8 u (2 + |gate|) of the value; each other step adds a few u of its terms.
"""
import numpy as np
import pytest
import torch

from oracle import feedforward as ff
from oracle import nodewise as nw
from tests.gpu_helpers import note
from tests.test_gpu_nodewise import COL_TERMS, COLS, DTYPES, EPS, ROW_TERMS, U, check_forward, close, f64, rows, tensor

pytestmark = pytest.mark.gpu
KINDS = ("f32", "bf16", "f16")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _etpc():
    import equivariant_gnn_tensor_amd as etpc
    return etpc


def params(rng, cols):
    return [tensor(v) for v in (1 + 0.3 * rng.standard_normal(cols), 0.3 * rng.standard_normal(cols), rng.standard_normal(cols),
                                rng.standard_normal(cols), rng.standard_normal(cols))]


def check_join_forward(y, h, stats, x, gate, res, w1, b1, scale, w2, b2, kind):
    n, mean, rstd = nw.layer_norm(x, w1, b1, EPS)
    top = np.abs(x).max(1)
    close(stats[:, 0], mean, ROW_TERMS * top, "mean")
    rel = ROW_TERMS + (ROW_TERMS * top * rstd) ** 2
    close(stats[:, 1], rstd, rel * rstd, "rstd")
    err = np.abs(w1) * (rstd * ROW_TERMS * top)[:, None] + (rel[:, None] + ROW_TERMS) * np.abs(n - b1) + ROW_TERMS * np.abs(b1)
    p, gerr = (1.0, 0.0) if gate is None else (1 / (1 + np.exp(-gate)), 8 * U * (2 + np.abs(gate)))
    rh = res + scale * p * n
    h_err = np.abs(scale * p) * (err + (gerr + 4 * U) * (np.abs(n - b1) + np.abs(b1))) + 2 * U * np.abs(res)
    if h is not None:
        close(h, rh, h_err, "h", kind)
    check_forward(y, stats[:, 2].contiguous(), stats[:, 3].contiguous(), rh, 2 * h_err.max(1), w2, b2, kind)


def check_join_backward(bars, x, gate, h, y_bar, h_bar, stats, w1, b1, scale, w2, kind):
    ref = ff.norm_gate_add_norm_backward(x, gate, h, y_bar, h_bar, stats, w1, b1, scale, w2)
    mean, rstd, mean_h, rstd_h = (v[:, None] for v in stats.T)
    hh, xh = (h - mean_h) * rstd_h, (x - mean) * rstd
    g2 = y_bar * w2
    ed = ROW_TERMS * (rstd_h * (np.abs(g2) + np.abs(g2).mean(1, keepdims=True) + np.abs(hh) * np.abs(g2 * hh).mean(1, keepdims=True))
                      + np.abs(h_bar))
    d = ref[2]
    p, gerr = (np.ones_like(x), 0.0) if gate is None else (1 / (1 + np.exp(-gate)), 8 * U * (2 + np.abs(gate)))
    m, em = xh * w1 + b1, 8 * U * (np.abs(xh * w1) + np.abs(b1))
    u = d * scale * p
    eu = np.abs(scale * p) * ed + (gerr + 4 * U) * np.abs(u)
    g1, eg = u * w1, np.abs(w1) * eu
    ex = rstd * (eg + eg.mean(1, keepdims=True) + np.abs(xh) * (eg * np.abs(xh)).mean(1, keepdims=True)
                 + ROW_TERMS * (np.abs(g1) + np.abs(g1).mean(1, keepdims=True) + np.abs(xh) * np.abs(g1 * xh).mean(1, keepdims=True)))
    q = 1.0 if gate is None else 1 / (1 + np.exp(gate))
    col = lambda terms, errors: COL_TERMS * np.abs(terms).sum(0) + errors.sum(0)  # noqa: E731
    bounds = (ex, q * (np.abs(m) * eu + np.abs(u) * em + (gerr + 4 * U) * np.abs(u * m)), ed, col(u * xh, eu * np.abs(xh)), col(u, eu),
              col(d * p * m, np.abs(p) * (np.abs(m) * ed + np.abs(d) * em + gerr * np.abs(d * m))), col(y_bar * hh, 0 * hh),
              col(y_bar, 0 * hh))
    names = ("x_bar", "gate_bar", "residual_bar", "w1_bar", "b1_bar", "scale_bar", "w2_bar", "b2_bar")
    for got, want, bound, name in zip(bars, ref, bounds, names):
        assert got is not None or want is None, name
        if got is not None:
            close(got, want, bound, name, kind if name in names[:3] else "f32")


def run_case(rng, n, cols, kind, gated, pitch=0):
    etpc = _etpc()
    x, res, yb, hb = (rows(rng, n, cols, kind, cols + pitch, shift=s) for s in (0.5, -0.2, 0.0, 0.1))
    gate = rows(rng, n, cols, kind, cols + pitch, shift=0.0) if gated else None
    w1, b1, scale, w2, b2 = params(rng, cols)
    y, h, stats = etpc.etpc_norm_gate_add_norm(x, gate, res, w1, b1, scale, w2, b2, eps=EPS)
    g = None if gate is None else f64(gate)
    check_join_forward(y, h, stats, f64(x), g, f64(res), f64(w1), f64(b1), f64(scale), f64(w2), f64(b2), kind)
    bars = etpc.etpc_norm_gate_add_norm_backward(x, h, yb, stats, gate, w1, b1, scale, w2, hb)
    check_join_backward(bars, f64(x), g, f64(h), f64(yb), f64(hb), f64(stats), f64(w1), f64(b1), f64(scale), f64(w2), kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 3, 70])
def test_join(kind, n):
    rng = np.random.default_rng(300 + n)
    for k, cols in enumerate(COLS):
        note(f"gated join {kind} rows={n} cols={cols}")
        run_case(rng, n, cols, kind, gated=k % 3 != 2, pitch=(0, 8, 5)[k % 3])


@pytest.mark.parametrize("kind,n,cols", [("f32", 5000, 64), ("bf16", 3001, 577), ("f16", 2500, 1024), ("f32", 20011, 3),
                                         ("bf16", 1100, 4104), ("f16", 3000, 1), ("f32", 300, 16400), ("bf16", 700, 8192)])
def test_join_many_rows(kind, n, cols):
    """More rows than workgroups: groups walk several rows and the column sums take two stages."""
    note(f"gated join {kind} rows={n} cols={cols}")
    run_case(np.random.default_rng(n), n, cols, kind, gated=True)
