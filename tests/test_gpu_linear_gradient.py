"""GPU checks of how exact the dense layer's gradient is, against oracle/feedforward.py (float64).

Steps, sums and activations count as in tests/test_gpu_linear.py.  Between narrow rows a 16-bit z_bar enters both
products as a rounded number and the rounded rest: off by half a step of the rest, which is half a step of z_bar
(2^-16 in bf16, 2^-22 in fp16, there at least half the smallest number, 2^-25).
"""
import numpy as np
import pytest
import torch
from scipy import special

from oracle import feedforward as ff
from tests.gpu_helpers import note
from tests.test_gpu_linear import DTYPES, HALF, KINDS, LEAST, U, check_backward, close, f64, matrix, steps, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _etpc():
    import equivariant_gnn_tensor_amd as etpc
    return etpc


NARROW = ((1, 8, 8), (1000, 8, 1), (300, 64, 1), (64, 33, 17), (129, 128, 32), (70, 32, 64), (1, 64, 64), (5000, 64, 64), (40, 61, 59),
          (2000, 5, 3), (33, 127, 31))


@pytest.mark.parametrize("act", ["silu", "gelu", "tanh", "relu"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_narrow_gradient_is_rounded_once(kind, act):
    etpc = _etpc()
    for k, (rows, n_in, n_out) in enumerate(NARROW):
        note(f"narrow gradient {kind} {act} {rows}x{n_in}->{n_out}")
        rng = np.random.default_rng(k)
        x, w = matrix(rng, rows, n_in, kind, 3, shift=0.3), weights(rng, n_in, n_out, kind, ("io", "oi")[k % 2])
        y_bar, z = matrix(rng, rows, n_out, kind, 1, shift=0.1), matrix(rng, rows, n_out, kind)
        x_bar, w_bar, _ = etpc.etpc_linear_backward(x, w, y_bar, z=z, act=act)
        x, w, y_bar, z = f64(x), f64(w), f64(y_bar), f64(z)
        rx, rw, _ = ff.linear_backward(x, w, y_bar, z, act)
        z_bar = np.abs(y_bar * ff.slope(z, act))
        dz = 32 * U * (1 + np.abs(z)) * np.abs(y_bar) + HALF[kind] ** 2 * z_bar + LEAST[kind]
        close(x_bar, rx, (steps(n_out) * (z_bar + dz) + dz) @ np.abs(w).T, "x_bar", kind)
        close(w_bar, rw, np.abs(x).T @ (steps(rows) * (z_bar + dz) + dz), "w_bar", kind)


def test_narrow_gradient_past_fp16():
    """z_bar past fp16's largest number, products within it; and infinities, which stay what the formula makes of them."""
    etpc = _etpc()
    rows, n_in, n_out = 40, 16, 8
    x = torch.full((rows, n_in), 2.0 ** -10, dtype=torch.float16, device="cuda")
    w = torch.full((n_in, n_out), 2.0 ** -5, dtype=torch.float16, device="cuda")
    y_bar = torch.full((rows, n_out), 64000.0, dtype=torch.float16, device="cuda")
    z = torch.full((rows, n_out), 1.5, dtype=torch.float16, device="cuda")
    x_bar, w_bar, b_bar = etpc.etpc_linear_backward(x, w, y_bar, z=z, act="gelu")
    z_bar = 64000 * float(ff.slope(1.5, "gelu"))
    assert z_bar > 65504
    tol = HALF["f16"] + 64 * U
    for got, ref in ((x_bar, n_out * z_bar / 32), (w_bar, rows * z_bar / 1024), (b_bar, rows * z_bar)):
        assert float((got.double() / ref - 1).abs().max()) <= tol
    for kind in ("bf16", "f16"):
        x, w, z = (t.to(DTYPES[kind]) for t in (x, w, z))
        y_bar = torch.ones(rows, n_out, device="cuda", dtype=DTYPES[kind])
        y_bar[3, 2] = -float("inf")
        x_bar, w_bar, b_bar = etpc.etpc_linear_backward(x, w, y_bar, z=z, act="gelu")
        keep = [k for k in range(rows) if k != 3]
        assert torch.isneginf(x_bar[3]).all() and torch.isfinite(x_bar[keep]).all()
        keep = [k for k in range(n_out) if k != 2]
        assert torch.isneginf(w_bar[:, 2]).all() and torch.isfinite(w_bar[:, keep]).all()
        assert torch.isneginf(b_bar[2]) and torch.isfinite(b_bar[keep]).all()


def terms(z, act):
    """Magnitudes that the slope is the sum of: an error relative to them is one that does not come from cancelling."""
    if act == "tanh":
        return ff.slope(z, act)
    if act == "silu":
        p = special.expit(z)
        return p + np.abs(z) * p * special.expit(-z)
    return special.ndtr(z) + np.abs(z) * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)


@pytest.mark.parametrize("act", ["silu", "gelu", "tanh"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_in", [8, 200])
def test_slopes_far_out(kind, act, n_in):
    """b_bar of one row is y_bar act'(z), unrounded: relative errors over all of z's useful range, between narrow rows
    and wider ones.  exp's argument is off by 2 u of itself (2 |z|, |z|, z^2 / 2) and its functions by some u."""
    etpc = _etpc()
    z = torch.arange(-96, 97, device="cuda") / 8.0
    for rows in (1, 40):
        cols = (z if n_in > 128 else z[::4]).contiguous().to(DTYPES[kind])
        zs = cols.expand(rows, -1)
        x = torch.zeros(rows, n_in, dtype=DTYPES[kind], device="cuda")
        w = torch.zeros(n_in, cols.numel(), dtype=DTYPES[kind], device="cuda")
        _, _, b_bar = etpc.etpc_linear_backward(x, w, torch.full_like(zs, 0.5).contiguous(), z=zs, act=act)
        v = f64(cols)
        bound = U * (32 + 4 * np.abs(v) + 4 * v * v * (act == "gelu")) * terms(v, act) + steps(rows) * np.abs(ff.slope(v, act))
        close(b_bar / (0.5 * rows), ff.slope(v, act), bound, "slope")


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("pitch", [0, 3])
@pytest.mark.parametrize("kind", KINDS)
def test_every_narrow_gradient(kind, pitch, act):
    """One, two and four tiles of 32 columns on either side, whole pieces and odd ones, with and without a slope, each
    output also on its own."""
    etpc = _etpc()
    for rows, n_in, n_out in ((300, 32, 32), (1001, 32, 64), (333, 64, 32), (33001, 64, 64), (32800, 128, 32), (77, 61, 31)):
        note(f"narrow gradient {kind} {act} {rows}x{n_in}->{n_out} pitch={pitch}")
        rng = np.random.default_rng(rows + pitch)
        x, w = matrix(rng, rows, n_in, kind, pitch, shift=0.3), weights(rng, n_in, n_out, kind, "oi", pitch)
        y_bar, z = matrix(rng, rows, n_out, kind, pitch, shift=0.1), matrix(rng, rows, n_out, kind, pitch)
        z = z if act != "none" else None
        bars = etpc.etpc_linear_backward(x, w, y_bar, z=z, act=act)
        check_backward(*bars, f64(x), f64(w), f64(y_bar), None if z is None else f64(z), act, kind)
        for k, name in enumerate("xwb"):
            assert torch.equal(etpc.etpc_linear_backward(x, w, y_bar, z=z, act=act, want=(name,))[k], bars[k])
