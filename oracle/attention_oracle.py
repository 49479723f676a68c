"""Float64 CPU oracle of the attention operators: the rotation and the cache
values an append leaves, and causal attention with its log-sum-exp. Plain and
slow; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

from . import fpformats as F


def rotate_f32(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x fp32 [..., D] rotated over its first 2 * len(cos) elements, one fp32
    rounding per operation (numpy's float32 arithmetic)."""
    x = x.astype(np.float32)
    y = x.copy()
    half = cos.shape[-1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def cache_codes(y: np.ndarray, scale: float) -> np.ndarray:
    """E4M3 codes an append stores for fp32 values y."""
    return F.fp32_to_e4m3_code((y.astype(np.float32) / np.float32(scale)).astype(np.float32))


def attention_rows(q, k, v, positions, scale):
    """q float64 [n, heads, D] at `positions` [n]; k, v [m, kv_heads, D].
    Row i attends to the positions 0 .. positions[i] (nothing if negative).
    Returns (o, lse, spread): o [n, heads, D], lse [n, heads], and `spread`
    = (sum_j w_j |v_j| / sum_j w_j, max_j scale sum_d |q_d k_jd|), from which
    tests derive what roundings may do."""
    n, heads, d = q.shape
    m, kv_heads = k.shape[:2]
    group = heads // kv_heads
    o, mean_abs = np.zeros((n, heads, d)), np.zeros((n, heads, d))
    lse, mag = np.full((n, heads), -np.inf), np.zeros((n, heads))
    positions = np.asarray(positions)
    live = positions >= 0
    if m == 0 or not live.any():
        return o, lse, (mean_abs, mag)
    seen = np.arange(m)[None, :] <= positions[live, None]
    for h in range(heads):
        qh, kh, vh = q[live, h], k[:, h // group], v[:, h // group]
        x = np.where(seen, scale * (qh @ kh.T), -np.inf)
        top = x.max(1, keepdims=True)
        w = np.exp(x - top)
        s = w.sum(1, keepdims=True)
        o[live, h] = (w @ vh) / s
        mean_abs[live, h] = (w @ np.abs(vh)) / s
        lse[live, h] = (top + np.log(s))[:, 0]
        mag[live, h] = np.where(seen, abs(scale) * (np.abs(qh) @ np.abs(kh).T), 0.0).max(1)
    return o, lse, (mean_abs, mag)
