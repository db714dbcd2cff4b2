"""Feed-forward operators in float64: the dense layer with its activations, the gated join of two
norms, the gradient norm.

TEST INFRASTRUCTURE ONLY: imported by ``tests/``, never by the product path.

Gradients are the closed formulas, pinned against finite differences by
tests/test_oracle_feedforward.py.
"""
from __future__ import annotations

import numpy as np
from scipy import special

from oracle.nodewise import layer_norm, layer_norm_backward

ACTS = ("none", "relu", "silu", "gelu", "tanh")


def act(z, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "silu":
        return z * special.expit(z)
    if name == "gelu":
        return z * special.ndtr(z)
    return np.tanh(z) if name == "tanh" else z


def slope(z, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name == "relu":
        return np.where(z > 0, 1.0, 0.0)
    if name == "silu":
        p = special.expit(z)
        return p + z * p * special.expit(-z)
    if name == "gelu":
        return special.ndtr(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    return np.cosh(np.clip(z, -300, 300)) ** -2.0 if name == "tanh" else np.ones_like(z)


def linear(x, w, b=None, residual=None, name: str = "none"):
    """(y, z)."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64) + (0.0 if b is None else b)
    y = act(z, name)
    return (y if residual is None else y + residual), z


def linear_backward(x, w, y_bar, z=None, name: str = "none"):
    """(x_bar, w_bar, b_bar)."""
    z_bar = y_bar * slope(z, name) if name != "none" else np.asarray(y_bar, np.float64)
    return z_bar @ w.T, x.T @ z_bar, z_bar.sum(0)


def _gate(gate, like):
    return np.ones_like(like) if gate is None else special.expit(gate)


def norm_gate_add_norm(x, gate, residual, w1, b1, scale, w2, b2, eps):
    """(y, h, stats): n = norm(x) w1 + b1, h = residual + scale sigmoid(gate) n, y = norm(h) w2 + b2."""
    n, mean, rstd = layer_norm(x, w1, b1, eps)
    h = residual + scale * _gate(gate, x) * n
    y, mean_h, rstd_h = layer_norm(h, w2, b2, eps)
    return y, h, np.stack((mean, rstd, mean_h, rstd_h), 1)


def norm_gate_add_norm_backward(x, gate, h, y_bar, h_bar, stats, w1, b1, scale, w2):
    """(x_bar, gate_bar, residual_bar, w1_bar, b1_bar, scale_bar, w2_bar, b2_bar)."""
    mean, rstd, mean_h, rstd_h = stats.T
    d, w2_bar, b2_bar = layer_norm_backward(h, y_bar, mean_h, rstd_h, w2)
    d = d + h_bar
    n = (x - mean[:, None]) * rstd[:, None] * w1 + b1
    p = _gate(gate, x)
    u = d * scale * p
    x_bar, w1_bar, b1_bar = layer_norm_backward(x, u, mean, rstd, w1)
    gate_bar = None if gate is None else u * n * special.expit(-gate)
    return x_bar, gate_bar, d, w1_bar, b1_bar, (d * p * n).sum(0), w2_bar, b2_bar


def grad_norm(grads, ord=2) -> float:
    grads = [np.asarray(g, np.float64) for g in grads if np.size(g)]
    if ord == 2:
        return float(np.sqrt(sum((g * g).sum() for g in grads)))
    return float(max((np.abs(g).max() for g in grads), default=0.0))


def clip_factor(norm: float, max_norm: float) -> float:
    """1 for a norm that fp32 does not hold as a finite number."""
    if not abs(norm) <= float(np.finfo(np.float32).max):
        return 1.0
    return min(1.0, max_norm / (norm + 1e-6))
