"""Oracle: rotary position embedding of a step's query and key rows, float64 numpy.

TEST INFRASTRUCTURE (see the package docstring): nothing in the CUDA library uses this file.

Element pairs (x, y) of a head's first rot_dim elements become (x c - y s, x s + y c) with the
cosine and sine of the pair's angle at the row's position: written here as a product of complex
numbers.  The table gives the angles' cosines and sines per position.
"""
from __future__ import annotations

import numpy as np

from .paged_attention import OracleError


def pairs(rot_dim: int, interleaved: bool) -> list[tuple[int, int]]:
    """Indices of the two elements of each pair of a head."""
    if rot_dim < 2 or rot_dim % 2:
        raise OracleError(f"rot_dim must be even, got {rot_dim}")
    half = rot_dim // 2
    return [(2 * j, 2 * j + 1) if interleaved else (j, j + half) for j in range(half)]


def rotate(x: np.ndarray, positions: np.ndarray, cos_sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x float64 [T, H, D] with each head rotated by row positions[t] of cos_sin [max_pos, rot_dim]."""
    x = np.array(x, dtype=np.float64)
    rot = cos_sin.shape[1]
    if rot > x.shape[2]:
        raise OracleError("rot_dim exceeds the head dim")
    rows = cos_sin[np.asarray(positions)].astype(np.float64)
    z = rows[:, :rot // 2] + 1j * rows[:, rot // 2:]
    for j, (a, b) in enumerate(pairs(rot, interleaved)):
        w = (x[:, :, a] + 1j * x[:, :, b]) * z[:, j][:, None]
        x[:, :, a], x[:, :, b] = w.real, w.imag
    return x


def positions_of(cu_seqlens_q: np.ndarray, kv_lens: np.ndarray) -> np.ndarray:
    """Absolute position of every packed token: kv_len - q_len + i for token i of its sequence."""
    out = []
    for s in range(len(kv_lens)):
        n = int(cu_seqlens_q[s + 1] - cu_seqlens_q[s])
        out += [int(kv_lens[s]) - n + i for i in range(n)]
    return np.array(out, dtype=np.int64)


def table(max_positions: int, rot_dim: int, base: float = 10000.0) -> np.ndarray:
    """fp32 [max_positions, rot_dim]: cosines then sines of position * base^(-2j / rot_dim)."""
    freq = float(base) ** (-np.arange(0, rot_dim, 2, dtype=np.float64) / rot_dim)
    ang = np.arange(max_positions, dtype=np.float64)[:, None] * freq
    return np.concatenate((np.cos(ang), np.sin(ang)), axis=1).astype(np.float32)
