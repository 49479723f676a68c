"""Helpers of the attention tests: seeded batches over a paged cache whose
unused rows hold NaN, the oracle's answer, and the bounds the arithmetic
allows."""
from __future__ import annotations

import numpy as np
import torch

import precision_gemm_token_gb300 as E
from oracle import attention_oracle as AO
from oracle import fpformats as F
from precision_gemm_token_gb300 import attention as A


def f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """seqs: (new tokens, tokens with them) of each sequence."""

    def __init__(self, seqs, heads, kv_heads, dim, fmt="bf16", page=16, order="head", seed=0, tail=0, spare=3,
                 table_extra=0, k_std=1.0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.heads, self.kv_heads, self.dim, self.fmt, self.page = seqs, heads, kv_heads, dim, fmt, page
        new = [n for n, _ in seqs]
        self.tokens = sum(new) + tail
        self.starts = [0] + list(np.cumsum(new)) if new else [0]
        self.q_start = torch.tensor(self.starts, dtype=torch.int32)
        self.kv_len = torch.tensor([m for _, m in seqs], dtype=torch.int32)
        held = [-(-m // page) for _, m in seqs]
        width = max(held, default=0) + table_extra
        pages = sum(held) + spare
        order_of = torch.randperm(pages, generator=g)[:sum(held)].tolist()
        # entries that no token needs hold an index far outside the pool
        self.table = torch.full((len(seqs), width), 1 << 30, dtype=torch.int32)
        for b, c in enumerate(held):
            self.table[b, :c] = torch.tensor([order_of.pop() for _ in range(c)], dtype=torch.int32)
        self.k_scale = self.v_scale = None
        if fmt == "e4m3":
            self.k_scale = 0.01 + 0.02 * torch.rand(kv_heads, generator=g)
            self.v_scale = 0.01 + 0.02 * torch.rand(kv_heads, generator=g)
        shape = (pages, kv_heads, page, dim) if order == "head" else (pages, page, kv_heads, dim)
        pools, self.rows = [], []
        for std, scale in ((k_std, self.k_scale), (1.0, self.v_scale)):
            x = torch.randn((pages, kv_heads, page, dim), generator=g) * std
            if fmt == "e4m3":
                c = torch.from_numpy(F.fp32_to_e4m3_code((x / scale[None, :, None, None]).numpy()))
                v = torch.from_numpy(F.e4m3_decode(c.numpy())) * scale.double()[None, :, None, None]
                nan = torch.full_like(c, 0x7F)
            else:
                c = x.to(torch.bfloat16)
                v = c.double()
                nan = torch.full_like(c, float("nan"))
            filled = nan
            for b, (_, m) in enumerate(seqs):
                for i, pg in enumerate(self.table[b, :held[b]].tolist()):
                    r = min(page, m - i * page)
                    filled[pg, :, :r] = c[pg, :, :r]
            # [tokens, kv_heads, dim] of each sequence, float64
            self.rows.append([v[self.table[b, :held[b]].long()].transpose(1, 2).reshape(-1, kv_heads, dim)[:m].numpy()
                              for b, (_, m) in enumerate(seqs)])
            pool = torch.empty(shape, dtype=c.dtype)
            view = pool if order == "head" else pool.transpose(1, 2)
            view.copy_(filled)
            pools.append(pool.to(device) if order == "head" else pool.to(device).transpose(1, 2))
        self.cache = A.PagedKVCache(*pools, *(s if s is None else s.to(device) for s in (self.k_scale, self.v_scale)))
        self.q = torch.randn(self.tokens, heads, dim, generator=g).to(torch.bfloat16)
        self.device = device

    def dev(self, *names):
        return [getattr(self, n).to(self.device) for n in names]

    def positions(self):
        """Position of each packed token, -1 where there is none."""
        pos = np.full(self.tokens, -1)
        for (n, m), t in zip(self.seqs, self.starts):
            pos[t:t + n] = np.maximum(np.arange(m - n, m), -1)
        return pos

    def oracle(self, scale):
        q, pos = f64(self.q), self.positions()
        o, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
        mean_abs, mag = np.zeros(q.shape), np.zeros(q.shape[:2])
        for b, ((n, _), t) in enumerate(zip(self.seqs, self.starts)):
            s = slice(t, t + n)
            o[s], lse[s], (mean_abs[s], mag[s]) = AO.attention_rows(q[s], self.rows[0][b], self.rows[1][b], pos[s],
                                                                    scale)
        return o, lse, mean_abs, mag

    def attend(self, **kw):
        kw.setdefault("max_new", max((n for n, _ in self.seqs), default=0))
        q, start, length, table = self.dev("q", "q_start", "kv_len", "table")
        return A.paged_attention(q, self.cache, start, length, table, **kw)


# unit roundoffs: bf16 has 8 significant bits (1 + 2^-8 lies halfway between
# the neighbours 1 and 1 + 2^-7), fp16 has 11
BF16_U, FP16_U = 2.0 ** -8, 2.0 ** -11


def out_bound(o, mean_abs, mag, weight_u):
    """|O - o| allowed: the output's rounding to bf16, the weights' rounding
    to the tensor cores' operand type (weight_u of the weighted mean of |v|),
    and the fp32 scores: each of up to 128 products and sums within 2^-24 of
    the score's magnitude, 2^-17 of it in all, which moves a weight by as much
    relative to the others on both sides of the quotient (2^-16), besides
    2^-14 for the exponentials and the fp32 sums of up to 2^9 roundings."""
    return BF16_U * np.abs(o) + (weight_u + 2.0 ** -16 * mag[..., None] + 2.0 ** -14) * mean_abs + 1e-30


def lse_bound(lse, mag):
    """Scores within 2^-17 of their magnitude, sums of weights within 2^-14,
    the logarithm's own rounding."""
    return 2.0 ** -17 * mag + 2.0 ** -14 + 2.0 ** -20 * np.abs(np.where(np.isfinite(lse), lse, 0.0))


def assert_attention(o_gpu, lse_gpu, o, lse, mean_abs, mag, what="", fmt="bf16"):
    got, bound = f64(o_gpu), out_bound(o, mean_abs, mag, FP16_U if fmt == "e4m3" else BF16_U)
    err = np.abs(got - o)
    assert np.isfinite(got).all(), (what, np.argwhere(~np.isfinite(got))[:5])
    assert (err <= bound).all(), (what, np.argwhere(err > bound)[:5], float((err / bound).max()))
    if lse_gpu is not None:
        got = f64(lse_gpu)
        empty = np.isneginf(lse)
        assert (np.isneginf(got) == empty).all(), what
        err = np.abs(np.where(empty, 0.0, got) - np.where(empty, 0.0, lse))
        b = lse_bound(lse, mag)
        assert (err <= b).all(), (what, float((err / b).max()))


def status_buf():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ensure_lib():
    E.build()
    E.load()
