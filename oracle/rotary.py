"""CPU oracle for rotary positions.

TEST INFRASTRUCTURE ONLY, plain numpy in float64.

Definition: with f_j the angle per position of pair j, the pair (a, b) of a token
at position p becomes amplitude * (a cos - b sin, b cos + a sin) of p * f_j; pairs
are (j, j + n/2) or (2j, 2j + 1) of the n dims from `first` on.
"""
from __future__ import annotations

import numpy as np


def frequencies(n: int, theta: float, kind=None, factor=1.0, original=0.0, fast=32.0, slow=1.0) -> np.ndarray:
    if kind == "base":
        theta = theta * factor ** (n / (n - 2))
    out = []
    for j in range(n // 2):
        f = theta ** (-2 * j / n)
        if kind == "linear":
            f = f / factor
        if kind == "parts":
            turns = original * f / (2 * np.pi)
            g = 1.0 if turns >= fast else 0.0 if turns <= slow else (turns - slow) / (fast - slow)
            f = f * g + f / factor * (1 - g)
        out.append(f)
    return np.array(out)


def rotate(x: np.ndarray, pos: np.ndarray, f: np.ndarray, first: int, interleaved: bool, amplitude=1.0) -> np.ndarray:
    """x [T, H, D] at positions pos [T]."""
    y = x.astype(np.float64)
    h = len(f)
    a = first + (2 * np.arange(h) if interleaved else np.arange(h))
    b = a + (1 if interleaved else h)
    c = amplitude * np.cos(pos[:, None] * f)[:, None]
    s = amplitude * np.sin(pos[:, None] * f)[:, None]
    u, w = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - w * s, w * c + u * s
    return y
