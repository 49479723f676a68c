"""Float64 CPU oracle of the operators in 8-bit blocks and of a mixture of
experts: block quantizer, block-scaled product, routing, the experts' gated
MLPs. Plain and slow; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

from . import fpformats as F

BLOCK = 128
AMAX_FLOOR = np.float32(1e-12)


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def quant_rows(x: np.ndarray):
    """x float32 [M, K] -> codes uint8 [M, K], scale float32 [blocks, M]."""
    x = np.asarray(x, np.float32)
    m, k = x.shape
    codes, scale = np.zeros((m, k), np.uint8), np.zeros((blocks(k), m), np.float32)
    for b in range(blocks(k)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        scale[b] = np.maximum(np.abs(part).max(1), AMAX_FLOOR) / np.float32(448)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = F.fp32_to_e4m3_code((part / scale[b][:, None]).astype(np.float32))
    return codes, scale


def quant_weight(w: np.ndarray):
    """w float32 [N, K] -> codes uint8 [N, K], scale float32 [blocks(N), blocks(K)]."""
    w = np.asarray(w, np.float32)
    n, k = w.shape
    codes, scale = np.zeros((n, k), np.uint8), np.zeros((blocks(n), blocks(k)), np.float32)
    for i in range(blocks(n)):
        for b in range(blocks(k)):
            at = np.s_[i * BLOCK:(i + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK]
            scale[i, b] = np.maximum(np.abs(w[at]).max(), AMAX_FLOOR) / np.float32(448)
            codes[at] = F.fp32_to_e4m3_code((w[at] / scale[i, b]).astype(np.float32))
    return codes, scale


def values_rows(codes, scale):
    """float64 [M, K] of codes and scale [blocks, M]."""
    k = codes.shape[1]
    return F.e4m3_decode(codes) * np.repeat(np.asarray(scale, np.float64).T, BLOCK, axis=1)[:, :k]


def values_weight(codes, scale):
    n, k = codes.shape
    s = np.repeat(np.repeat(np.asarray(scale, np.float64), BLOCK, axis=0)[:n], BLOCK, axis=1)[:, :k]
    return F.e4m3_decode(codes) * s


def product(a, w):
    """(a w^T, |a| |w|^T) of float64 values; rows with NaN poison only themselves."""
    with np.errstate(invalid="ignore"):
        return a @ w.T, np.abs(a) @ np.abs(w).T


def route(logits, top, bias=None, scoring="softmax", groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    """ids int32 [T, top] and weights float64 [T, top], token by token."""
    z = np.asarray(logits, np.float64)
    tokens, n = z.shape
    ids, weights = np.full((tokens, top), -1, np.int32), np.zeros((tokens, top))
    size = n // groups
    for t in range(tokens):
        l = z[t].copy()
        l[np.isnan(l)] = -np.inf
        l = np.minimum(l, np.float64(np.finfo(np.float32).max))
        here = l > -np.inf
        if bias is not None:
            b = np.asarray(bias, np.float64)
            here &= ~np.isnan(b) & (b > -np.inf)
        score = np.zeros(n)
        there = l > -np.inf
        if there.any():
            if scoring == "softmax":
                e = np.exp(l[there] - l[there].max())
                score[there] = e / e.sum()
            else:
                with np.errstate(over="ignore"):
                    score[there] = 1 / (1 + np.exp(-l[there]))
        c = score + (0 if bias is None else b)
        c[~here] = -np.inf
        # without a bias the order of the scores is that of the logits, which 64 bits may not show
        order = np.where(here, l if bias is None else c, -np.inf)
        if groups > 1:
            if bias is None and group_best == 1:
                value = order.reshape(groups, size).max(1)
            else:
                s = -np.sort(-c.reshape(groups, size), 1)[:, :group_best]
                value = np.where(s[:, 0] > -np.inf, np.where(s > -np.inf, s, 0).sum(1), -np.inf)
            kept = np.argsort(-value, kind="stable")[:top_groups]
            out = np.ones(groups, bool)
            out[kept] = False
            order[np.repeat(out, size)] = -np.inf
        # (of choices that 64 bits cannot tell apart the larger logit first)
        chosen = [e for e in np.lexsort((-l, -order))[:top] if order[e] > -np.inf]
        ids[t, :len(chosen)] = chosen
        if not chosen:
            continue
        s = score[chosen]
        if renormalize:
            # in proportion, where the scores themselves may be too small for 64 bits
            log = l[chosen] if scoring == "softmax" else -np.logaddexp(0, -l[chosen])
            s = np.exp(log - log.max())
            s = s / s.sum()
        weights[t, :len(chosen)] = s * scale
    return ids, weights


def silu(g):
    with np.errstate(over="ignore", invalid="ignore"):
        return g / (1 + np.exp(-g))
