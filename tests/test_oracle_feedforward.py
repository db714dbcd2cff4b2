"""Pins of oracle/feedforward.py (CPU): gradients against finite differences, closed values."""
import numpy as np
import pytest

from oracle import feedforward as ff
from tests.test_oracle_nodewise import _differences


@pytest.mark.parametrize("name", ff.ACTS)
def test_slopes(name):
    z = np.linspace(-6, 6, 97) + 0.011   # not at relu's corner
    step = 1e-5
    d = (ff.act(z + step, name) - ff.act(z - step, name)) / (2 * step)
    assert np.abs(d - ff.slope(z, name)).max() < 1e-8


def test_closed_values():
    assert ff.act(1.0, "silu") == pytest.approx(1 / (1 + np.exp(-1)), abs=1e-15)
    assert ff.act(1.0, "gelu") == pytest.approx(0.8413447460685429, abs=1e-15)
    assert ff.act(-1.0, "relu") == 0 and ff.slope(0.0, "relu") == 0 and ff.slope(0.0, "tanh") == 1


@pytest.mark.parametrize("name", ff.ACTS)
def test_linear_gradients(name):
    rng = np.random.default_rng(5)
    x, w, b = rng.standard_normal((4, 3)), rng.standard_normal((3, 5)), rng.standard_normal(5)
    res, y_bar = rng.standard_normal((4, 5)), rng.standard_normal((4, 5))
    y, z = ff.linear(x, w, b, res, name)
    grads = ff.linear_backward(x, w, y_bar, z, name)
    f = lambda x, w, b, r: (ff.linear(x, w, b, r, name)[0] * y_bar).sum()  # noqa: E731
    numeric = (_differences(lambda v: f(v, w, b, res), x), _differences(lambda v: f(x, v, b, res), w),
               _differences(lambda v: f(x, w, v, res), b), _differences(lambda v: f(x, w, b, v), res))
    for got, ref in zip((*grads, y_bar), numeric):
        assert np.abs(got - ref).max() < 1e-8


@pytest.mark.parametrize("gated", [True, False])
def test_join_gradients(gated):
    rng = np.random.default_rng(6)
    n, c = 3, 7
    x, res, y_bar, h_bar = (rng.standard_normal((n, c)) for _ in range(4))
    gate = rng.standard_normal((n, c)) if gated else None
    params = [rng.standard_normal(c) for _ in range(5)]

    def f(x, gate, res, w1, b1, scale, w2, b2):
        y, h, _ = ff.norm_gate_add_norm(x, gate, res, w1, b1, scale, w2, b2, 1e-5)
        return (y * y_bar).sum() + (h * h_bar).sum()
    args = [x, gate, res, *params]
    _, h, stats = ff.norm_gate_add_norm(*args, 1e-5)
    w1, b1, scale, w2, _ = params
    grads = ff.norm_gate_add_norm_backward(x, gate, h, y_bar, h_bar, stats, w1, b1, scale, w2)
    for k, got in enumerate(grads):
        if args[k] is None:
            assert got is None
            continue
        ref = _differences(lambda v: f(*args[:k], v, *args[k + 1:]), args[k])
        assert np.abs(got - ref).max() < 1e-7, k


def test_norm_and_factor():
    grads = [np.array([3.0, 0.0]), np.zeros(0), np.array([[-4.0]])]
    assert ff.grad_norm(grads) == 5.0 and ff.grad_norm(grads, np.inf) == 4.0 and ff.grad_norm([]) == 0.0
    assert ff.clip_factor(5.0, 2.5) == pytest.approx(0.5, abs=1e-6) and ff.clip_factor(5.0, 10.0) == 1.0
    assert ff.clip_factor(np.inf, 1.0) == 1.0 and ff.clip_factor(np.nan, 1.0) == 1.0
