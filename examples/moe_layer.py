"""A mixture-of-experts layer with its weights in 8-bit blocks, as a decoder
layer calls it after its attention: the router's logits, the choice of experts
(sigmoid scores, a bias that balances them, groups), the experts' gated MLPs,
and a shared expert beside them; eager, and as one captured graph for decoding.

    python examples/moe_layer.py [--tokens N]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import precision_gemm_token_gb300 as E  # noqa: E402
from precision_gemm_token_gb300 import blocks as B  # noqa: E402
from precision_gemm_token_gb300 import moe as M  # noqa: E402


class MoeLayer:
    """hidden -> hidden; random weights. The shared expert is an expert of its own that every token takes."""

    def __init__(self, hidden=1024, inner=512, experts=16, top=4, groups=4, top_groups=2, scale=2.5, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *shape: (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).to(  # noqa: E731
            torch.bfloat16)
        self.top, self.groups, self.top_groups, self.scale = top, groups, top_groups, scale
        self.router = rnd(experts, hidden).float()
        self.bias = 0.05 * torch.randn(experts, generator=g, device="cuda")
        self.experts = M.quantize_experts(rnd(experts, inner, hidden), rnd(experts, inner, hidden), rnd(experts, hidden, inner))
        self.shared = M.quantize_experts(rnd(1, inner, hidden), rnd(1, inner, hidden), rnd(1, hidden, inner))
        self.ws = B.BlockWorkspace("cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def route(self, x):
        logits = x.float() @ self.router.T
        return M.route(logits, self.top, bias=self.bias, scoring="sigmoid", groups=self.groups, top_groups=self.top_groups,
                       group_best=2, scale=self.scale)

    def __call__(self, x):
        """x bf16 [tokens, hidden] -> bf16 [tokens, hidden]"""
        ids, weights = self.route(x)
        y = M.experts(x, ids, weights, self.experts, workspace=self.ws, status=self.status)
        everybody = torch.zeros(x.shape[0], 1, dtype=torch.int32, device="cuda")
        return y + M.experts(x, everybody, torch.ones(x.shape[0], 1, device="cuda"), self.shared, workspace=self.ws,
                             status=self.status)


class Decoder:
    """The layer for a fixed number of tokens, captured once: step() copies the rows in and replays."""

    def __init__(self, layer, tokens, hidden):
        self.x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
        layer(self.x)                                       # (the workspace at its size before the capture)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = layer(self.x)

    def step(self, x):
        self.x[:x.shape[0]].copy_(x)
        self.graph.replay()
        return self.y[:x.shape[0]]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=500)
    a = ap.parse_args()
    E.build()
    layer = MoeLayer()
    prompt = torch.randn(a.tokens, 1024, device="cuda").to(torch.bfloat16)
    y = layer(prompt)
    dec = Decoder(layer, 8, 1024)
    for n in (1, 5, 8):
        off = (dec.step(prompt[:n]).float() - y[:n].float()).abs().max() / y.float().abs().max()
        print(f"{n} tokens decoded: off the prompt's by {off.item():.1e} of its largest")
    torch.cuda.synchronize()
    t0 = time.time()
    for _ in range(100):
        dec.step(prompt[:8])
    torch.cuda.synchronize()
    print(f"decode step of 8 tokens: {(time.time() - t0) * 1e4:.1f} us; status {int(layer.status)}")


if __name__ == "__main__":
    main()
