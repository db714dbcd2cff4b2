"""Node-wise operators in float64: dropout masks, layer norm, residual join, irreps norm.

TEST INFRASTRUCTURE ONLY: imported by ``tests/``, never by the product path.

Masks come from Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers:
as easy as 1, 2, 3", SC 2011).  Gradients are the closed formulas.

Pinned by tests/test_oracle_nodewise.py: the generator's published known answers, finite
differences of every forward map against its gradient, and rotations of irreps features.
"""
from __future__ import annotations

from typing import Sequence, Tuple

import numpy as np

Irrep = Tuple[int, int, int]
_MASK = np.uint64(0xFFFFFFFF)
_HIGH = np.uint64(32)


def philox4x32(counter, key):
    """Ten rounds.  counter: four broadcastable arrays of 32-bit words, key: two words."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> _HIGH) ^ c[1] ^ np.uint64(k[0]), b & _MASK, (a >> _HIGH) ^ c[3] ^ np.uint64(k[1]), a & _MASK]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.broadcast_arrays(*c)


def threshold(p: float) -> int:
    return int(np.rint(65536.0 * p))


def keep_fields(rows: int, groups: int, p: float, seed: int, offset: int) -> np.ndarray:
    """bool [rows, 8 groups]: field c mod 8 of counter (c div 8, row, offset) is kept."""
    w = philox4x32((np.arange(groups)[None, :], np.arange(rows)[:, None], offset & 0xFFFFFFFF, offset >> 32),
                   (seed & 0xFFFFFFFF, seed >> 32))
    f = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], axis=-1)
    return f.reshape(rows, 8 * groups) >= threshold(p)


def _scale(p: float) -> float:
    t = threshold(p)
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def dropout(x, p: float, seed: int, offset: int) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    keep = keep_fields(rows, (cols + 7) // 8, p, seed, offset)[:, :cols]
    return np.where(keep, x * _scale(p), 0.0)


def blocks(irreps: Sequence[Irrep]):
    """(mul, l, parity, offset in a row, first channel, first bias or None) per block."""
    out, off, ch, bias = [], 0, 0, 0
    for mul, l, parity in irreps:
        scalar = l == 0 and parity == 1
        out.append((mul, l, parity, off, ch, bias if scalar else None))
        off += mul * (2 * l + 1)
        ch += mul
        bias += mul if scalar else 0
    return out


def irreps_dropout(x, irreps: Sequence[Irrep], p: float, seed: int, offset: int) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    rows = x.shape[0]
    keep = keep_fields(rows, sum((b[0] + 7) // 8 for b in irreps), p, seed, offset)
    y, group = np.zeros_like(x), 0
    for mul, l, _, off, _, _ in blocks(irreps):
        m = keep[:, 8 * group:8 * group + mul]
        for mu in range(2 * l + 1):
            part = slice(off + mu * mul, off + (mu + 1) * mul)
            y[:, part] = np.where(m, x[:, part] * _scale(p), 0.0)
        group += (mul + 7) // 8
    return y


def layer_norm(x, w, b, eps: float):
    """(y, mean, rstd) of rows; w and b are vectors."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    return d * rstd[:, None] * w + b, mean, rstd


def layer_norm_backward(x, y_bar, mean, rstd, w):
    """(x_bar, w_bar, b_bar) with the forward pass's statistics."""
    xh = (np.asarray(x, dtype=np.float64) - mean[:, None]) * rstd[:, None]
    g = y_bar * w
    x_bar = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True))
    return x_bar, (y_bar * xh).sum(axis=0), y_bar.sum(axis=0)


def irreps_norm(x, irreps: Sequence[Irrep], w, b, eps: float):
    """(y, stats [N, blocks, 2]) of ir_mul features."""
    x = np.asarray(x, dtype=np.float64)
    y, stats = np.zeros_like(x), np.zeros((x.shape[0], len(irreps), 2))
    for k, (mul, l, _, off, ch, bias) in enumerate(blocks(irreps)):
        part = slice(off, off + mul * (2 * l + 1))
        v = x[:, part]
        mean = v.mean(axis=1) if l == 0 else np.zeros(x.shape[0])
        d = v - mean[:, None]
        rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
        y[:, part] = d * rstd[:, None] * np.tile(w[ch:ch + mul], 2 * l + 1)
        if bias is not None:
            y[:, part] += b[bias:bias + mul]
        stats[:, k, 0], stats[:, k, 1] = mean, rstd
    return y, stats


def irreps_norm_backward(x, y_bar, stats, irreps: Sequence[Irrep], w):
    """(x_bar, w_bar, b_bar) with the forward pass's statistics."""
    x, y_bar = np.asarray(x, dtype=np.float64), np.asarray(y_bar, dtype=np.float64)
    x_bar, w_bar, b_bar = np.zeros_like(x), [], []
    for k, (mul, l, _, off, ch, bias) in enumerate(blocks(irreps)):
        part = slice(off, off + mul * (2 * l + 1))
        rstd = stats[:, k, 1][:, None]
        xh = (x[:, part] - stats[:, k, 0][:, None]) * rstd
        g = y_bar[:, part] * np.tile(w[ch:ch + mul], 2 * l + 1)
        t = g - xh * (g * xh).mean(axis=1, keepdims=True)
        if l == 0:
            t -= g.mean(axis=1, keepdims=True)
        x_bar[:, part] = rstd * t
        w_bar.append((y_bar[:, part] * xh).sum(axis=0).reshape(2 * l + 1, mul).sum(axis=0))
        if bias is not None:
            b_bar.append(y_bar[:, part].sum(axis=0))
    cat = lambda v: np.concatenate(v) if v else np.zeros(0)  # noqa: E731
    return x_bar, cat(w_bar), cat(b_bar)
