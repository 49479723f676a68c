"""A multi-tenant attention layer served end to end: one fused q/k/v projection
(a slice and an adapter pair each), the append to a paged cache, the attention
over it, and the output projection, for steps that mix decoding sequences with
chunks of new prompts.

    python examples/attention_layer.py [--kv bf16|e4m3] [--decode N]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import precision_gemm_token_gb300 as E  # noqa: E402
from precision_gemm_token_gb300 import attention as A  # noqa: E402
from precision_gemm_token_gb300 import tensors as T  # noqa: E402


def rotary_table(positions, dim, base=500000.0, device="cuda"):
    """fp32 [positions, dim]: cosines, then sines."""
    t = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return torch.cat([t.cos(), t.sin()], 1).float().to(device)


class AttentionLayer:
    """hidden -> hidden; weights and adapters are random. step() takes any mix
    of sequences: each brings its new tokens, one or many."""

    def __init__(self, hidden=1024, heads=8, kv_heads=2, dim=128, tenants=4, rank=16, pages=512, page=16,
                 positions=4096, kv="bf16", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *shape, std: (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
        self.hidden, self.heads, self.kv_heads, self.dim, self.page = hidden, heads, kv_heads, dim, page
        n = (heads + 2 * kv_heads) * dim
        self.slice_end = [heads * dim, (heads + kv_heads) * dim, n]
        self.w_qkv = T.quantize_weight(rnd(n, hidden, std=hidden ** -0.5), E.FMT_FP8)
        self.w_o = T.quantize_weight(rnd(hidden, heads * dim, std=(heads * dim) ** -0.5), E.FMT_FP8)
        self.a_qkv, self.b_qkv = rnd(tenants, 3 * rank, hidden, std=hidden ** -0.5), rnd(tenants, n, rank, std=0.1)
        self.a_o, self.b_o = rnd(tenants, rank, heads * dim, std=(heads * dim) ** -0.5), rnd(tenants, hidden, rank, std=0.1)
        pool = (pages, page, kv_heads, dim)             # token-major; the cache takes any strides
        if kv == "bf16":
            k, v = (torch.zeros(pool, dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in range(2))
            self.cache = A.PagedKVCache(k, v)
        else:
            k, v = (torch.zeros(pool, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in range(2))
            scale = torch.full((kv_heads,), 1 / 16, dtype=torch.float32, device="cuda")
            self.cache = A.PagedKVCache(k, v, scale, scale)
        self.table_cs = rotary_table(positions, dim)
        self.proj_ws, self.attn_ws = T.LayerWorkspace("cuda"), A.AttentionWorkspace("cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # the host's side of the cache
        self.free = list(range(pages))
        self.pages, self.length = {}, {}

    def qkv(self, x, tenant):
        y = T.layer_forward_slices(x, self.w_qkv, self.a_qkv, self.b_qkv, tenant, self.slice_end,
                                   workspace=self.proj_ws, status=self.status)
        y = y.view(x.shape[0], -1, self.dim)
        return y[:, :self.heads], y[:, self.heads:self.heads + self.kv_heads], y[:, self.heads + self.kv_heads:]

    def plan(self, seqs):
        """(q_start, kv_len, page table, most new tokens) of a step; seqs: (name, new tokens)."""
        rows, starts, lens = [], [0], []
        for name, new in seqs:
            mine, held = self.pages.setdefault(name, []), self.length.get(name, 0) + new
            while len(mine) * self.page < held:
                mine.append(self.free.pop())
            self.length[name] = held
            rows.append(mine)
            starts.append(starts[-1] + new)
            lens.append(held)
        width = max(len(r) for r in rows)
        dev = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
        return dev(starts), dev(lens), dev([r + [0] * (width - len(r)) for r in rows]), max(n for _, n in seqs)

    def step(self, x, tenant, plan):
        """x bf16 [tokens, hidden], packed as planned; tenant int32 [tokens]. Enqueues five calls."""
        starts, lens, table, most = plan
        q, k, v = self.qkv(x, tenant)
        q = A.kv_append(q, k, v, self.cache, starts, lens, table, self.table_cs, q_out=q, status=self.status)
        o = A.paged_attention(q, self.cache, starts, lens, table, max_new=most, workspace=self.attn_ws,
                              status=self.status)
        return T.layer_forward(o.view(x.shape[0], -1), self.w_o, self.a_o, self.b_o, tenant, workspace=self.proj_ws,
                               status=self.status), q, o

    def release(self, name):
        self.free += self.pages.pop(name)
        del self.length[name]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--kv", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--decode", type=int, default=32)
    args = ap.parse_args()
    E.build()
    layer = AttentionLayer(kv=args.kv)
    prompts = {"a": 500, "b": 37, "c": 211}
    tenant_of = {"a": 0, "b": 3, "c": -1, "d": 2}      # -1: the base weights alone

    def run(seqs):
        tenant = torch.tensor([tenant_of[s] for s, n in seqs for _ in range(n)], dtype=torch.int32).cuda()
        x = torch.randn(tenant.numel(), layer.hidden, device="cuda").to(torch.bfloat16)
        return layer.step(x, tenant, layer.plan(seqs))[0]

    run(list(prompts.items()))                         # three prompts in one step
    run([("a", 1), ("b", 1), ("c", 1), ("d", 300)])    # they decode while a fourth prompt comes in
    layer.release("b")
    seqs = [("a", 1), ("c", 1), ("d", 1)]
    run(seqs)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(args.decode):
        y = run(seqs)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) * 1e3 / max(args.decode, 1)
    assert int(layer.status.item()) == 0 and bool(torch.isfinite(y).all())
    print(f"kv {args.kv}: lengths {layer.length}, {ms:.3f} ms per decode step with its host work")


if __name__ == "__main__":
    main()
