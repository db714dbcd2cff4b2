"""Pins of oracle/nodewise.py (CPU): the generator's published known answers, gradients
against finite differences, equivariance, and the masks' statistics."""
import numpy as np
import pytest

from oracle import nodewise as nw
from oracle.wigner import random_rotation, wigner_d

EPS = 1e-5
IRREPS = [(3, 0, 1), (2, 0, -1), (4, 1, -1), (2, 2, 1), (1, 3, -1), (2, 0, 1)]
DIM = sum(m * (2 * l + 1) for m, l, _ in IRREPS)
CHANNELS, BIASES = sum(m for m, _, _ in IRREPS), 5


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_known_answers(counter, key, words):
    assert tuple(int(v) for v in nw.philox4x32(counter, key)) == words


def test_mask_statistics():
    """The share kept is 1 - T / 65536 to five deviations, rows and offsets do not repeat."""
    p, n = 0.3, 64 * 4096
    a, b = nw.keep_fields(64, 512, p, 7, 0), nw.keep_fields(64, 512, p, 7, 1)
    q = 1 - nw.threshold(p) / 65536
    for m in (a, b):
        assert abs(m.mean() - q) < 5 * np.sqrt(q * (1 - q) / n)
    both = q * q + (1 - q) * (1 - q)
    assert abs((a == b).mean() - both) < 5 * np.sqrt(both * (1 - both) / n)
    assert abs((a[:-1] == a[1:]).mean() - both) < 5 * np.sqrt(both * (1 - both) / (n - 4096))
    assert nw.keep_fields(4, 4, 0.0, 1, 2).all() and not nw.keep_fields(4, 4, 1.0, 1, 2).any()


def _differences(f, x, step=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += step
        down[i] -= step
        g[i] = (f(up) - f(down)) / (2 * step)
    return g


# central differences: h^2 f''' / 6 and rounding / h, both under 1e-8 for these sizes of order one
FD_TOL = 1e-7


def test_layer_norm_gradient():
    rng = np.random.default_rng(1)
    x, yb = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    w, b = rng.standard_normal(7), rng.standard_normal(7)
    _, mean, rstd = nw.layer_norm(x, w, b, EPS)
    xb, wb, bb = nw.layer_norm_backward(x, yb, mean, rstd, w)
    assert np.abs(xb - _differences(lambda t: (yb * nw.layer_norm(t, w, b, EPS)[0]).sum(), x)).max() < FD_TOL
    assert np.abs(wb - _differences(lambda t: (yb * nw.layer_norm(x, t, b, EPS)[0]).sum(), w)).max() < FD_TOL
    assert np.abs(bb - _differences(lambda t: (yb * nw.layer_norm(x, w, t, EPS)[0]).sum(), b)).max() < FD_TOL


def test_irreps_norm_gradient():
    rng = np.random.default_rng(2)
    x, yb = rng.standard_normal((2, DIM)), rng.standard_normal((2, DIM))
    w, b = rng.standard_normal(CHANNELS), rng.standard_normal(BIASES)
    _, stats = nw.irreps_norm(x, IRREPS, w, b, EPS)
    xb, wb, bb = nw.irreps_norm_backward(x, yb, stats, IRREPS, w)
    f = lambda x_, w_, b_: (yb * nw.irreps_norm(x_, IRREPS, w_, b_, EPS)[0]).sum()  # noqa: E731
    assert np.abs(xb - _differences(lambda t: f(t, w, b), x)).max() < FD_TOL
    assert np.abs(wb - _differences(lambda t: f(x, t, b), w)).max() < FD_TOL
    assert np.abs(bb - _differences(lambda t: f(x, w, t), b)).max() < FD_TOL


def rotate(x, R, improper):
    """ir_mul features under the rotation R (times the inversion when improper)."""
    y = np.empty_like(x)
    for mul, l, parity, off, _, _ in nw.blocks(IRREPS):
        part = slice(off, off + mul * (2 * l + 1))
        D = wigner_d(l, R) * (parity if improper else 1)
        y[:, part] = np.einsum("ab,nbc->nac", D, x[:, part].reshape(-1, 2 * l + 1, mul)).reshape(x.shape[0], -1)
    return y


@pytest.mark.parametrize("improper", [False, True])
def test_irreps_operators_are_equivariant(improper):
    rng = np.random.default_rng(3)
    x, R = rng.standard_normal((4, DIM)), random_rotation(rng)
    w, b = rng.standard_normal(CHANNELS), rng.standard_normal(BIASES)
    for f in (lambda t: nw.irreps_norm(t, IRREPS, w, b, EPS)[0], lambda t: nw.irreps_dropout(t, IRREPS, 0.4, 5, 6)):
        assert np.abs(f(rotate(x, R, improper)) - rotate(f(x), R, improper)).max() < 1e-12


def test_scalar_blocks_are_a_layer_norm():
    rng = np.random.default_rng(4)
    x, w, b = rng.standard_normal((5, 9)), rng.standard_normal(9), rng.standard_normal(9)
    y, mean, rstd = nw.layer_norm(x, w, b, EPS)
    z, stats = nw.irreps_norm(x, [(9, 0, 1)], w, b, EPS)
    assert np.array_equal(y, z) and np.array_equal(stats[:, 0], np.stack([mean, rstd], 1))
