"""Experts' outputs kept in fp32 until their weighted sum: Y is rounded once, as the formula in 64 bits allows."""
import numpy as np
import pytest
import torch

import precision_gemm_token_gb300 as E
from oracle import fpformats as F
from oracle import moe_oracle as O
from precision_gemm_token_gb300 import blocks as B
from precision_gemm_token_gb300 import moe as M
from tests import moe_util as U

pytestmark = pytest.mark.gpu
F32 = torch.float32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def expected(hq, hs, ids, weights, d, ds):
    """(y, its bound): sums of a product's terms and of the experts in fp32, then one rounding to bf16."""
    T, top = ids.shape
    h = O.values_rows(hq.reshape(T * top, -1), hs).reshape(T, top, -1)
    y, bound, size = (np.zeros((T, d.shape[1])) for _ in range(3))
    for e in range(d.shape[0]):
        t, j = np.nonzero(ids == e)
        if len(t) == 0:
            continue
        p, ps = O.product(h[t, j], O.values_weight(d[e], ds[e]))
        w = weights[t, j].astype(np.float64)[:, None]
        np.add.at(y, t, w * p)
        np.add.at(bound, t, np.abs(w) * U.sum_bound(h.shape[2], ps))
        np.add.at(size, t, np.abs(w * p))
    bound += top * 2.0 ** -23 * size
    return y, bound + U.BF16 * (np.abs(y) + bound)


def choices(t, top, e, seed, gone):
    g = np.random.default_rng(seed)
    ids = np.argsort(g.standard_normal((t, e)) + 1.5 * g.standard_normal(e), 1)[:, :top].astype(np.int32)
    ids[g.random((t, top)) < 0.05] = -1
    if gone:
        ids[-gone:] = -1
    return ids, g.uniform(-1.0, 1.0, (t, top)).astype(np.float32)


# tokens, top, experts, hidden, inner, tokens without an expert
SIZES = [(1, 1, 1, 16, 16, 0), (1, 8, 16, 512, 256, 0), (3, 2, 4, 144, 112, 1), (64, 4, 16, 640, 384, 3),
         (300, 2, 3, 256, 128, 5), (130, 8, 60, 2064, 144, 0), (700, 1, 2, 384, 272, 0), (20, 17, 33, 96, 48, 2)]


@pytest.mark.parametrize("t,top,e,hidden,inner,gone", SIZES)
def test_down(t, top, e, hidden, inner, gone):
    ids, weights = choices(t, top, e, t, gone)
    hq, hs = O.quant_rows(U.activations(t * top, inner, seed=t).float().numpy())
    w = U.expert_weights(e, inner, hidden, seed=200)
    none = (ids < 0).reshape(-1)
    hq[none], hs[:, none] = 0x7F, np.nan                # NaN where nobody looks
    given = [dev(a) for a in (hq.reshape(t, top, inner), hs, ids, weights)]
    experts = M.ExpertWeights(*map(dev, w))
    y = M.experts_down(*given, experts, parts=F32)
    hq[none], hs[:, none] = 0, 0
    want, bound = expected(hq, hs, ids, weights, w[2], w[3])
    U.close(U.f64(y), want, bound)
    # in one call with its up half, of a workspace that the bf16 form has left its own in
    x, ws = U.activations(t, hidden, seed=t + 1).cuda(), B.BlockWorkspace("cuda")
    M.experts(x, given[2], given[3], experts, workspace=ws)
    both = M.experts(x, given[2], given[3], experts, workspace=ws, parts=F32)
    up = M.experts_up(x, given[2], experts)
    assert torch.equal(both, M.experts_down(*up, given[2], given[3], experts, parts=F32, workspace=ws))


def test_one_rounding_alone():
    """Whole numbers whose sums are exact in 32 bits, of both signs: the rounded sum itself, and not a sum of roundings."""
    g = np.random.default_rng(4)
    t, top, e, hidden, inner = 200, 3, 5, 400, 272
    h = g.integers(-3, 4, (t, top, inner)).astype(np.float64)
    d = g.integers(-3, 4, (e, hidden, inner)).astype(np.float64)
    ids, _ = choices(t, top, e, 9, 0)
    weights = g.choice([-1.0, 1.0], (t, top)).astype(np.float32)
    one = lambda *shape: np.ones(shape, np.float32)  # noqa: E731
    w = M.ExpertWeights(torch.zeros(e, 2, inner, hidden, dtype=torch.uint8).cuda(),
                        torch.zeros(e, 2, O.blocks(inner), O.blocks(hidden)).cuda(), dev(F.fp32_to_e4m3_code(d)),
                        dev(one(e, O.blocks(hidden), O.blocks(inner))))
    args = dev(F.fp32_to_e4m3_code(h)), dev(one(O.blocks(inner), t * top)), dev(ids), dev(weights), w
    want, rounded = np.zeros((t, hidden)), torch.zeros(t, hidden)
    for j in range(top):
        part = np.where(ids[:, j, None] >= 0, np.einsum("ti,thi->th", h[:, j], d[ids[:, j]]), 0) * weights[:, j, None]
        want += part
        rounded += torch.from_numpy(part).to(torch.bfloat16).float()
    want = torch.from_numpy(want).to(torch.bfloat16)
    assert torch.equal(M.experts_down(*args, parts=F32).cpu(), want)
    # (and the form in bf16 is what it was)
    y = M.experts_down(*args).cpu()
    assert torch.equal(y, rounded.to(torch.bfloat16)) and not torch.equal(y, want)


def test_captured_and_on_another_stream():
    t, top, e, hidden, inner = 40, 4, 6, 256, 144
    w = M.ExpertWeights(*map(dev, U.expert_weights(e, inner, hidden, seed=1)))
    x = U.activations(t, hidden, seed=2).cuda()
    ids, weights = (dev(a) for a in choices(t, top, e, 3, 2))
    ws = B.BlockWorkspace("cuda")
    want = M.experts(x, ids, weights, w, workspace=ws, parts=F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = M.experts(x, ids, weights, w, stream=side, parts=F32)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.zeros(t, hidden + 8, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.experts(x, ids, weights, w, out=out[:, :hidden], workspace=ws, parts=F32)
    for seed in (5, 6):
        x.copy_(U.activations(t, hidden, seed))
        graph.replay()
        assert torch.equal(out[:, :hidden], M.experts(x, ids, weights, w, parts=F32)) and (out[:, hidden:] == 0).all()


def test_refuses_other_types():
    w = M.ExpertWeights(*map(dev, U.expert_weights(2, 16, 32, seed=1)))
    x = torch.zeros(1, 32, dtype=torch.bfloat16, device="cuda")
    ids, weights = M.route(torch.zeros(1, 2, device="cuda"), 1)
    with pytest.raises(E.EpiloraError):
        M.experts(x, ids, weights, w, parts=torch.float16)
