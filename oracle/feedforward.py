"""Feed-forward operators in float64: the dense layer with its activations.

TEST INFRASTRUCTURE ONLY: imported by ``tests/``, never by the product path.

Gradients are the closed formulas, pinned against finite differences by
tests/test_oracle_feedforward.py.
"""
from __future__ import annotations

import numpy as np
from scipy import special

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
