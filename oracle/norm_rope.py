"""RMS norm of every head and rotation by position, and their gradient: fp64 CPU.

TEST INFRASTRUCTURE ONLY, like the rest of the oracle: the library never imports it, and it shares no code
with the CUDA kernels.

For a row x of d values at position pos:
  u = x / sqrt(mean(x^2) + eps) * w,   y = R_pos u,
where R_pos turns the pairs (a, b) of the first 2 * cos.shape[1] values:
  y_a = u_a cos - u_b sin,   y_b = u_b cos + u_a sin,
with pair i = (i, i + half), or (2i, 2i + 1) when interleaved. The gradient is written from the
row's Jacobian, dx = J^T dy, and pinned against differences of the forward in the tests.
"""
from __future__ import annotations

import numpy as np


def rotation_matrix(cos_row, sin_row, d: int, interleaved: bool) -> np.ndarray:
    """R_pos as a d x d matrix."""
    half = len(cos_row)
    R = np.eye(d)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        R[a, a], R[a, b] = cos_row[i], -sin_row[i]
        R[b, b], R[b, a] = cos_row[i], sin_row[i]
    return R


def _matrices(positions, cos, sin, d, interleaved):
    if cos is None:
        return {int(p): np.eye(d) for p in set(np.ravel(positions).tolist())}
    return {int(p): rotation_matrix(np.float64(cos[p]), np.float64(sin[p]), d, interleaved)
            for p in set(np.ravel(positions).tolist())}


def norm_rope(x, positions, w=None, eps: float = 1e-6, norm: bool = True, cos=None, sin=None, interleaved: bool = False):
    """x [T, heads, d] at positions [T]: y [T, heads, d]."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    u = x
    if norm:
        u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if w is not None:
            u = u * np.asarray(w, dtype=np.float64)
    R = _matrices(positions, cos, sin, d, interleaved)
    return np.stack([u[t] @ R[int(p)].T for t, p in enumerate(positions)]) if len(x) else u


def norm_rope_backward(x, dy, positions, w=None, eps: float = 1e-6, norm: bool = True, cos=None, sin=None,
                       interleaved: bool = False):
    """(dx [T, heads, d], dw [d]) for the output gradient dy."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    T, heads, d = x.shape
    wv = np.ones(d) if w is None else np.asarray(w, dtype=np.float64)
    R = _matrices(positions, cos, sin, d, interleaved)
    dx, dw = np.empty_like(x), np.zeros(d)
    for t, p in enumerate(positions):
        for h in range(heads):
            du = R[int(p)].T @ dy[t, h]
            if not norm:
                dx[t, h] = du
                continue
            a = np.sqrt((x[t, h] @ x[t, h]) / d + eps)
            J = np.eye(d) / a - np.outer(x[t, h], x[t, h]) / (d * a ** 3)   # of x / a, symmetric
            dx[t, h] = J @ (wv * du)
            dw += du * x[t, h] / a
    return dx, dw
