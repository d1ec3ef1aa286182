"""Plain CPU oracle of the rotary positions and of the norm before them, in
extended precision (angles of far positions need more than float64's product).

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

LD = np.longdouble


def norm(x, kind: str, norm_dim: int, weight, bias, eps: float) -> np.ndarray:
    """x [..., dim] with features [0, norm_dim) normed."""
    x = np.asarray(x, LD).copy()
    y = x[..., :norm_dim]
    if kind == "layer":
        y = y - y.mean(-1, keepdims=True)
    y = y / np.sqrt((y * y).mean(-1, keepdims=True) + LD(eps)) * np.asarray(weight, LD)
    if kind == "layer" and bias is not None:
        y = y + np.asarray(bias, LD)
    x[..., :norm_dim] = y
    return x


def rotate(x, positions, inv_freq, offset: int = 0, interleaved: bool = False, amplitude: float = 1.0,
           reverse: bool = False) -> np.ndarray:
    """x [tokens, heads, dim]; one pair at a time."""
    out = np.asarray(x, LD).copy()
    half = len(inv_freq)
    pos = np.asarray(positions).astype(LD)
    for i in range(half):
        ia, ib = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + i + half)
        ang = pos * LD(inv_freq[i]) * (-1 if reverse else 1)
        c, s = np.cos(ang)[:, None] * LD(amplitude), np.sin(ang)[:, None] * LD(amplitude)
        a, b = out[:, :, ia].copy(), out[:, :, ib].copy()
        out[:, :, ia], out[:, :, ib] = a * c - b * s, b * c + a * s
    return out
