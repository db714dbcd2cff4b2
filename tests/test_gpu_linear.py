"""GPU checks of the dense layer against oracle/feedforward.py (float64).

Tolerances, u = 2^-24.  Inputs reach the oracle exactly (already rounded to the element type).
Products of 16-bit numbers are exact in fp32, those of fp32 numbers round once inside the
multiply-add.  The matrix cores add the products of 2 (fp32) to 16 numbers of k to a running
sum; counted as K / 2 + 16 additions one after another with 2 u each, relative to the sum of
the products' magnitudes.  The sums of rows (w_bar, b_bar) count the same with K = rows.  An
activation follows an error of z with a slope below 1.2; its own error is some u of the value
times the condition of exp (|z|) or of the normal distribution's tail (z^2).  Where a 16-bit
z_bar enters the products it has been rounded once more (half a step of itself).  Each result is
rounded to its type once: half a step, 2^-8 (bf16), 2^-11 (fp16), 2^-24 (fp32) of the value.
"""
import numpy as np
import pytest
import torch

from oracle import feedforward as ff
from tests.gpu_helpers import note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -120, "bf16": 2.0 ** -120, "f16": 2.0 ** -24}
KINDS = ("f32", "bf16", "f16")
# rows, inputs, outputs: single numbers, below and past a vector, a slice of k, a tile, odd and even
SIZES = ((1, 1, 1), (1, 5, 3), (2, 8, 8), (3, 64, 64), (64, 7, 1), (70, 65, 33), (33, 32, 8), (129, 2047, 65), (257, 128, 200),
         (300, 64, 511), (5, 1024, 1024), (8, 200, 1000), (9, 1000, 72), (16, 520, 136), (500, 9, 17), (1000, 1, 64), (130, 72, 1),
         (17, 4100, 16))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _etpc():
    import equivariant_gnn_tensor_amd as etpc
    return etpc


def f64(t):
    return t.detach().double().cpu().numpy()


def matrix(rng, n, cols, kind, pitch=0, scale=1.0, shift=0.0):
    """A [n, cols] view of rows cols + pitch elements apart; every other element is NaN."""
    full = torch.full((n, cols + pitch), float("nan"), dtype=DTYPES[kind], device="cuda")
    full[:, :cols] = torch.from_numpy(scale * rng.standard_normal((n, cols)) + shift).to("cuda", DTYPES[kind])
    return full[:, :cols]


def weights(rng, n_in, n_out, kind, layout, pitch=0):
    if layout == "io":
        return matrix(rng, n_in, n_out, kind, pitch, n_in ** -0.5)
    return matrix(rng, n_out, n_in, kind, pitch, n_in ** -0.5).t()


def vector(rng, n):
    return torch.from_numpy(rng.standard_normal(n)).to("cuda", torch.float32)


def steps(k):
    return 2 * U * (k / 2 + 16)


def close(got, ref, bound, what, kind="f32"):
    """|got - ref| <= bound + the rounding of the result; equal where ref is not finite."""
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    tol = bound + HALF[kind] * (np.abs(ref) + bound) + LEAST[kind]
    bad = ~(np.abs(got - ref) <= tol) & np.isfinite(ref)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], np.broadcast_to(tol, ref.shape)[bad][:4])
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what


def act_error(z, y, name):
    """Of the activation itself at z, with result y."""
    return {"none": 0.0, "relu": 0.0, "silu": 16 * U * (1 + np.abs(z)) * np.abs(y), "gelu": 16 * U * (1 + z * z) * np.abs(y),
            "tanh": 16 * U * np.abs(y)}[name]


def check_forward(y, z, x, w, b, res, name, kind):
    ry, rz = ff.linear(x, w, b, res, name)
    dz = steps(x.shape[1]) * (np.abs(x) @ np.abs(w) + np.abs(b))
    if z is not None:
        close(z, rz, dz, "z", kind)
    plain = ff.act(rz, name)
    err = 1.2 * dz + act_error(np.abs(rz) + dz, np.abs(plain) + 1.2 * dz, name)
    close(y, ry, err + 4 * U * (np.abs(plain) + np.abs(ry)), "y", kind)


def check_backward(x_bar, w_bar, b_bar, x, w, y_bar, z, name, kind):
    rx, rw, rb = ff.linear_backward(x, w, y_bar, z, name)
    z_bar = y_bar * ff.slope(z, name) if name != "none" else y_bar
    own = 0.0 if name == "none" else 32 * U * (1 + np.abs(z)) * np.abs(y_bar)
    dz = own if name == "none" else own + HALF[kind] * np.abs(z_bar) + LEAST[kind]
    rows, n_out = y_bar.shape
    if x_bar is not None:
        close(x_bar, rx, (steps(n_out) * (np.abs(z_bar) + dz) + dz) @ np.abs(w).T, "x_bar", kind)
    if w_bar is not None:
        close(w_bar, rw, np.abs(x).T @ (steps(rows) * (np.abs(z_bar) + dz) + dz), "w_bar", kind)
    if b_bar is not None:
        close(b_bar, rb, (steps(rows) * np.abs(z_bar) + own).sum(0), "b_bar")


def run_case(seed, rows, n_in, n_out, kind, name, layout, pitch, residual=True):
    etpc = _etpc()
    note(f"linear {kind} {rows}x{n_in}->{n_out} {name} {layout} pitch={pitch}")
    rng = np.random.default_rng(seed)
    x, w, b = matrix(rng, rows, n_in, kind, pitch, shift=0.3), weights(rng, n_in, n_out, kind, layout, pitch), vector(rng, n_out)
    res = matrix(rng, rows, n_out, kind, pitch) if residual else None
    y, z = etpc.etpc_linear(x, w, b, residual=res, act=name)
    assert (z is None) == (name == "none")
    check_forward(y, z, f64(x), f64(w), f64(b), None if res is None else f64(res), name, kind)
    y_bar = matrix(rng, rows, n_out, kind, pitch, shift=0.1)
    x_bar, w_bar, b_bar = etpc.etpc_linear_backward(x, w, y_bar, z=z, act=name)
    assert w_bar.dtype == x.dtype and b_bar.dtype == torch.float32
    check_backward(x_bar, w_bar, b_bar, f64(x), f64(w), f64(y_bar), None if z is None else f64(z), name, kind)


@pytest.mark.parametrize("layout", ["io", "oi"])
@pytest.mark.parametrize("pitch", [0, 8, 5])
@pytest.mark.parametrize("kind", KINDS)
def test_linear(kind, pitch, layout):
    for k, (rows, n_in, n_out) in enumerate(SIZES):
        run_case(k, rows, n_in, n_out, kind, ff.ACTS[(k + pitch) % 5], layout, pitch, residual=k % 2 == 0)


@pytest.mark.parametrize("kind,rows,n_in,n_out,layout", [
    ("bf16", 5000, 64, 64, "io"), ("f16", 20011, 64, 64, "oi"), ("f32", 7001, 64, 64, "io"), ("bf16", 3000, 1024, 520, "oi"),
    ("f16", 4100, 512, 1032, "io"), ("f32", 2100, 264, 1000, "oi"), ("bf16", 30000, 8, 64, "io"), ("f16", 9000, 128, 16, "io"),
    ("bf16", 8200, 256, 2056, "io"), ("f16", 8200, 1032, 2056, "oi"), ("f32", 4097, 300, 511, "io"), ("f16", 4098, 264, 520, "oi")])
def test_linear_many_rows(kind, rows, n_in, n_out, layout):
    """More tiles than compute units, ranges of rows for the weight gradient, tiles that end outside."""
    run_case(rows, rows, n_in, n_out, kind, "silu", layout, 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,n_in,n_out,layout,pitch", [
    (65537, 64, 64, "io", 0), (65570, 128, 32, "oi", 8), (65600, 32, 128, "io", 5), (65551, 100, 60, "oi", 0),
    (65569, 60, 100, "io", 8), (65539, 33, 65, "oi", 5), (65568, 127, 64, "io", 0), (65536, 64, 64, "oi", 0),
    (65537, 128, 128, "io", 0), (66000, 17, 127, "oi", 0), (32769, 64, 64, "oi", 5), (32768, 128, 32, "io", 0)])
def test_linear_narrow_many_rows(kind, rows, n_in, n_out, layout, pitch):
    """On either side of where a narrow layer's rows are enough for a kernel that keeps its weights in LDS."""
    run_case(rows, rows, n_in, n_out, kind, ff.ACTS[1 + (n_in + n_out) % 4], layout, pitch)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,n_in,n_out", [(1, 300, 2100), (2, 2300, 4200), (1, 130, 8200), (2, 2049, 2048), (1, 17, 515)])
def test_linear_one_or_two_rows(kind, rows, n_in, n_out):
    """Either width of a workgroup's outputs, more inputs than one pass holds."""
    for layout in ("io", "oi"):
        run_case(rows + n_out, rows, n_in, n_out, kind, "silu", layout, 0)
