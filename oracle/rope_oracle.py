"""Float64 CPU oracle of the rotary positions (test infrastructure only): positions of the
token grid, per-head RMS norm, rotation of channel pairs, and their gradients, written
from the definitions in numpy. Shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def positions(grid, n_text=0, text_pos=None, origin=(0.0, 0.0, 0.0), step=(1.0, 1.0, 1.0)):
    """[N + n_text, 3] positions of the key sequence; NaN where a text row is not turned."""
    T, H, W = grid
    t, y, x = np.meshgrid(np.arange(T), np.arange(H), np.arange(W), indexing="ij")
    grid_pos = np.stack([t, y, x], -1).reshape(-1, 3) * np.asarray(step, np.float64) + np.asarray(origin, np.float64)
    text = np.full((n_text, 3), np.nan) if text_pos is None else np.asarray(text_pos, np.float64).reshape(n_text, 3)
    return np.concatenate([grid_pos, text], 0)


def angles(pos, axes, head_dim, theta):
    """[rows, head_dim / 2] angles: pair i of an axis with m channels turns by pos theta^(-2i/m)."""
    out = np.zeros((pos.shape[0], head_dim // 2))
    at = 0
    for a, m in enumerate(axes):
        for i in range(m // 2):
            out[:, at] = pos[:, a] * float(theta) ** (-2.0 * i / m)
            at += 1
    return np.nan_to_num(out, nan=0.0)


def split_pairs(x, pairs):
    """The two channels of every pair, each [..., head_dim / 2]."""
    half = x.shape[-1] // 2
    return (x[..., 0::2], x[..., 1::2]) if pairs == "adjacent" else (x[..., :half], x[..., half:])


def join_pairs(a, b, pairs):
    return np.stack([a, b], -1).reshape(*a.shape[:-1], 2 * a.shape[-1]) if pairs == "adjacent" else np.concatenate([a, b], -1)


def rotate(x, ang, pairs):
    a, b = split_pairs(x, pairs)
    c, s = np.cos(ang), np.sin(ang)
    return join_pairs(a * c - b * s, a * s + b * c, pairs)


def forward(x, ang, pairs, weight=None, eps=1e-6):
    """x [B, heads, rows, d], ang [rows, d/2] -> the normalised and rotated rows."""
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    return rotate(x, ang, pairs)


def backward(x, ang, pairs, dy, weight=None, eps=1e-6):
    """(dx, dweight) of sum(dy * forward(x)); dweight None without a weight."""
    g = rotate(dy, -ang, pairs)
    if weight is None:
        return g, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dweight = (g * xh).sum((0, 1, 2))
    g = g * weight
    return r * (g - xh * (g * xh).mean(-1, keepdims=True)), dweight
