"""Helpers of the tests of the operators in 8-bit blocks: seeded inputs, the
oracle's answers, and the bounds the arithmetic allows."""
from __future__ import annotations

import numpy as np
import torch

from oracle import fpformats as F
from oracle import moe_oracle as O

# Sums of a block's 128 products on the tensor cores and of the blocks after
# them, fp32: each addition loses at most one unit of 2^-23 (it may truncate)
# of the sum of the terms' sizes; the scales' product and its rounding three
# more. A rounding to bf16 moves a value by at most 2^-8 of it.
BF16, E4M3 = 2.0 ** -8, 2.0 ** -4


def sum_bound(k, size):
    return (O.BLOCK + O.blocks(k) + 3) * 2.0 ** -23 * size


def close(got, want, bound, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = np.isnan(want)
    assert (np.isnan(got) == nan).all(), what
    off = np.where(nan, 0, np.abs(got - want) - bound)
    assert (off <= 0).all(), f"{what}: {int((off > 0).sum())} of {off.size} beyond the bound, the worst by {off.max()}"


def f64(t):
    return t.detach().double().cpu().numpy()


def activations(m, k, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g) * torch.exp(0.5 * torch.randn(m, 1, generator=g))
    return (x * torch.exp(0.7 * torch.randn(k, generator=g))).to(torch.bfloat16)


def weight(n, k, seed):
    """(codes, scale) as numpy; blocks of unlike scale."""
    g = np.random.default_rng(seed)
    codes, scale = O.quant_weight(g.standard_normal((n, k)).astype(np.float32) * 0.02)
    return codes, (scale * g.uniform(0.5, 2.0, scale.shape)).astype(np.float32)


def expert_weights(e, inner, hidden, seed):
    made = [[weight(inner, hidden, seed + 3 * i), weight(inner, hidden, seed + 3 * i + 1), weight(hidden, inner, seed + 3 * i + 2)]
            for i in range(e)]
    gu = np.stack([np.stack([m[0][0], m[1][0]]) for m in made])
    gus = np.stack([np.stack([m[0][1], m[1][1]]) for m in made])
    return gu, gus, np.stack([m[2][0] for m in made]), np.stack([m[2][1] for m in made])


def up_expected(xq, xs, ids, gu, gus):
    """(h [T, top, inner], its bound) in float64; zero where there is no expert."""
    T, top = ids.shape
    inner = gu.shape[2]
    x = O.values_rows(xq, xs)
    h, bound = np.zeros((T, top, inner)), np.zeros((T, top, inner))
    for e in range(gu.shape[0]):
        t, j = np.nonzero(ids == e)
        if len(t) == 0:
            continue
        (g, gs), (u, us) = (O.product(x[t], O.values_weight(gu[e, p], gus[e, p])) for p in range(2))
        eg, eu = sum_bound(x.shape[1], gs), sum_bound(x.shape[1], us)
        s = O.silu(g)
        h[t, j] = s * u
        # |silu'| < 1.1; of silu itself the exponent's argument is rounded (|g| 2^-24 of the result), and the exponential,
        # the sum, the quotient and the product are off by less than 2^-20 together
        own = (2.0 ** -20 + np.abs(g) * 2.0 ** -24) * np.abs(h[t, j])
        bound[t, j] = 1.1 * eg * (np.abs(u) + eu) + (np.abs(s) + 1.1 * eg) * eu + own
    return h, bound


def check_quantized(codes, scale, h, bound, what=""):
    """Codes [T, top, inner] and scales against h within `bound` of where it was rounded."""
    T, top, inner = h.shape
    s = f64(scale).reshape(-1, T, top)
    for b in range(O.blocks(inner)):
        part = np.s_[:, :, b * O.BLOCK:(b + 1) * O.BLOCK]
        size, off = np.abs(h[part]).max(2), bound[part].max(2)
        there = size > 0
        want = np.where(there, np.maximum(size, 1e-12) / 448, s[b])
        close(s[b], want, off / 448 + 2.0 ** -22 * want, what + " scale")
        got = F.e4m3_decode(codes.cpu().numpy()[part]) * s[b][..., None]
        # half a step: 2^-4 of a normal code, 2^-10 of the scale below them; the quotient's rounding is far below both
        close(got, h[part], np.maximum(E4M3 * (np.abs(h[part]) + bound[part]), 2.0 ** -10 * s[b][..., None]) * (1 + 2.0 ** -20)
              + bound[part], what)


def down_expected(hq, hs, ids, weights, d, ds):
    T, top = ids.shape
    hidden = d.shape[1]
    h = O.values_rows(hq.reshape(T * top, -1), hs).reshape(T, top, -1)
    y, bound, size = np.zeros((T, hidden)), np.zeros((T, hidden)), np.zeros((T, hidden))
    for e in range(d.shape[0]):
        t, j = np.nonzero(ids == e)
        if len(t) == 0:
            continue
        p, ps = O.product(h[t, j], O.values_weight(d[e], ds[e]))
        w = weights[t, j].astype(np.float64)[:, None]
        off = sum_bound(h.shape[2], ps)
        np.add.at(y, t, w * p)
        # each expert's output is rounded to bf16 once
        np.add.at(bound, t, np.abs(w) * (off + BF16 * (np.abs(p) + off)))
        np.add.at(size, t, np.abs(w * p))
    bound += top * 2.0 ** -23 * size
    return y, bound + BF16 * (np.abs(y) + bound)
