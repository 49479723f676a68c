"""Routing and the experts' products on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from precision_gemm_token_gb300 import blocks as B
from precision_gemm_token_gb300 import moe as M
from tests import moe_util as U

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check_route(logits, top, **kw):
    ids, weights = M.route(logits, top, **kw)
    cpu = {k: (v.cpu().numpy() if torch.is_tensor(v) else v) for k, v in kw.items()}
    want, w = O.route(logits.float().cpu().numpy(), top, **cpu)
    assert np.array_equal(ids.cpu().numpy(), want), np.argwhere(ids.cpu().numpy() != want)[:4]
    # an exponential of an argument rounded to 2^-24 of it, sums of up to 40 additions, a quotient or two
    l = logits.float().cpu().numpy().astype(np.float64)
    span = np.nanmax(np.where(np.isfinite(l), np.abs(l), 0), initial=0, axis=1, keepdims=True) * 2
    U.close(U.f64(weights), w, np.abs(w) * (np.minimum(span, 200) + 64) * 2.0 ** -23 + 1e-37)
    return ids, weights


@pytest.mark.parametrize("fmt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 128, 8), (7, 5, 5), (33, 60, 4), (100, 64, 6), (50, 129, 32), (64, 256, 8),
                                   (40, 512, 10), (9, 1000, 8), (5, 1024, 32)])
def test_route(t, e, k, fmt):
    g = torch.Generator().manual_seed(t + e)
    logits = (2 * torch.randn(t, e, generator=g)).to(fmt).cuda()
    bias = 0.05 * torch.randn(e, generator=g).cuda()
    for scoring in ("softmax", "sigmoid"):
        for b in (None, bias):
            check_route(logits, k, scoring=scoring, bias=b, renormalize=b is None, scale=1.0 if b is None else 2.5)


@pytest.mark.parametrize("fmt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e,groups,kept,k", [(256, 8, 4, 8), (256, 8, 1, 8), (60, 4, 2, 6), (160, 8, 3, 6), (64, 32, 5, 7),
                                             (12, 3, 3, 12), (512, 16, 2, 16)])
def test_route_groups(e, groups, kept, k, fmt):
    g = torch.Generator().manual_seed(e + groups)
    logits = (1.5 * torch.randn(67, e, generator=g)).to(fmt).cuda()
    bias = 0.05 * torch.randn(e, generator=g).cuda()
    for scoring in ("softmax", "sigmoid"):
        for best in (1, 2):
            for b in (None, bias):
                check_route(logits, k, scoring=scoring, groups=groups, top_groups=kept, group_best=best, bias=b)


def test_route_many_tokens():
    """Some of them with two choices closer than 32 bits can tell."""
    g = torch.Generator().manual_seed(3)
    logits = (torch.randn(3000, 256, generator=g)).cuda()
    bias = 0.05 * torch.randn(256, generator=g).cuda()
    check_route(logits, 8, scoring="sigmoid", bias=bias, groups=8, top_groups=4, group_best=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_near_ties_go_by_the_exact_order(scoring):
    """Choices that differ by less than a 32-bit step of them: the bias takes back what the score adds, nearly."""
    g = np.random.default_rng(1)
    t, e = 64, 96
    logits = torch.from_numpy(g.standard_normal((t, e)).astype(np.float32))
    z = logits.double().numpy()[0]
    s = np.exp(z - z.max()) / np.exp(z - z.max()).sum() if scoring == "softmax" else 1 / (1 + np.exp(-z))
    bias = torch.from_numpy((1.0 - s).astype(np.float32))           # token 0: every choice is 1 within 2^-24
    logits[1:8] = logits[0]
    check_route(logits.cuda(), 9, scoring=scoring, bias=bias.cuda())
    check_route(logits.cuda(), 9, scoring=scoring, bias=bias.cuda(), groups=8, top_groups=3, group_best=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest_index(scoring):
    logits = torch.zeros(6, 64)
    logits[1, 40:] = 1
    logits[2, ::3] = -1
    logits[3] = 88.0
    logits[4] = -88.0
    logits[5, 5] = logits[5, 63] = 50.0
    for kw in ({}, dict(groups=8, top_groups=2, group_best=2), dict(groups=8, top_groups=2, group_best=1),
               dict(bias=torch.full((64,), 0.25).cuda())):
        check_route(logits.cuda(), 7, scoring=scoring, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kw", [{}, dict(groups=4, top_groups=2), dict(groups=4, top_groups=2, group_best=2), dict(bias=True),
                                dict(bias=True, groups=4, top_groups=2, group_best=2), dict(renormalize=False)])
def test_route_masked_logits(scoring, kw):
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(2)
    logits = torch.randn(12, 40, generator=g)
    logits[0] = -inf                                  # nobody left
    logits[1] = nan
    logits[2, 3:] = -inf                              # three left
    logits[3, ::2] = nan
    logits[4, 7] = inf
    logits[5, [3, 30]] = inf
    logits[6] = torch.finfo(torch.float32).min        # a mask of the lowest value: everybody alike
    logits[7, 1:] = torch.finfo(torch.float32).min
    logits[8] = torch.finfo(torch.float32).max
    logits[9, 10:] = -inf
    logits[10] -= 200                                 # scores of a sigmoid too small for 32 bits
    logits[11, 20:] -= 150
    kw = dict(kw)
    if kw.pop("bias", False):
        kw["bias"] = 0.1 * torch.randn(40, generator=g).cuda()
        kw["bias"][4] = -inf
        kw["bias"][5] = nan
    if not kw.get("renormalize", True):
        logits = logits[:10]
    check_route(logits.cuda(), 6, scoring=scoring, **kw)


def test_route_strided_rows_and_given_outputs():
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(30, 100, generator=g).cuda()
    logits = wide[:, 17:77]
    ids = torch.empty(30, 4, dtype=torch.int32, device="cuda")
    weights = torch.empty(30, 4, device="cuda")
    got = M.route(logits, 4, ids=ids, weights=weights)
    assert got[0] is ids and got[1] is weights
    want = M.route(logits.contiguous(), 4)
    assert torch.equal(ids, want[0]) and torch.equal(weights, want[1])


def choices(t, top, e, seed, gone=0):
    """Unlike numbers of tokens an expert; the last `gone` tokens have none, other slots lack one here and there."""
    g = np.random.default_rng(seed)
    liking = g.standard_normal((t, e)) + 1.5 * g.standard_normal(e)
    ids = np.argsort(-liking, 1)[:, :top].astype(np.int32)
    ids[g.random((t, top)) < 0.05] = -1
    if gone:
        ids[-gone:] = -1
    return ids, g.uniform(0.1, 1.0, (t, top)).astype(np.float32)


# tokens, top, experts, hidden, inner, tokens without an expert
MIXTURES = [(1, 1, 1, 16, 16, 0), (1, 8, 16, 512, 256, 0), (3, 2, 4, 144, 112, 1), (64, 4, 16, 640, 384, 3),
            (37, 3, 7, 1040, 208, 0), (300, 2, 3, 256, 128, 5), (130, 8, 60, 272, 144, 0), (700, 1, 2, 384, 272, 0)]


@pytest.mark.parametrize("t,top,e,hidden,inner,gone", MIXTURES)
def test_experts_up(t, top, e, hidden, inner, gone):
    ids, _ = choices(t, top, e, seed=t, gone=gone)
    x = U.activations(t, hidden, seed=t + 1)
    w = U.expert_weights(e, inner, hidden, seed=100)
    codes, scale = M.experts_up(x.cuda(), dev(ids), M.ExpertWeights(*map(dev, w)))
    h, bound = U.up_expected(*O.quant_rows(x.float().numpy()), ids, w[0], w[1])
    U.check_quantized(codes, scale, h, bound)
    none = torch.from_numpy(ids < 0)
    assert (codes.cpu()[none] == 0).all() and (scale.cpu().view(-1, t, top)[:, none] == 0).all()


@pytest.mark.parametrize("t,top,e,hidden,inner,gone", MIXTURES)
def test_experts_down(t, top, e, hidden, inner, gone):
    ids, weights = choices(t, top, e, seed=t, gone=gone)
    hq, hs = O.quant_rows(U.activations(t * top, inner, seed=t).float().numpy())
    hq[(ids < 0).reshape(-1)] = 0x7F                  # NaN where nobody looks
    hs[:, (ids < 0).reshape(-1)] = np.nan
    w = U.expert_weights(e, inner, hidden, seed=200)
    y = M.experts_down(dev(hq.reshape(t, top, inner)), dev(hs), dev(ids), dev(weights), M.ExpertWeights(*map(dev, w)))
    hq[(ids < 0).reshape(-1)] = 0
    hs[:, (ids < 0).reshape(-1)] = 0
    want, bound = U.down_expected(hq, hs, ids, weights, w[2], w[3])
    U.close(U.f64(y), want, bound)


@pytest.mark.parametrize("t,top,e,hidden,inner,gone", MIXTURES)
def test_experts_is_up_then_down(t, top, e, hidden, inner, gone):
    ids, weights = (dev(a) for a in choices(t, top, e, seed=t, gone=gone))
    x = U.activations(t, hidden, seed=t + 1).cuda()
    w = M.ExpertWeights(*map(dev, U.expert_weights(e, inner, hidden, seed=100)))
    ws = B.BlockWorkspace("cuda")
    y = M.experts(x, ids, weights, w, workspace=ws)
    h, hs = M.experts_up(x, ids, w)
    assert torch.equal(y, M.experts_down(h, hs, ids, weights, w, workspace=ws))
    assert torch.equal(y, M.experts(x, ids, weights, w, workspace=ws))


def test_experts_integers():
    """Whole numbers small enough that every sum is exact: the products of the right rows with the right weights."""
    g = np.random.default_rng(4)
    t, top, e, hidden, inner = 200, 2, 5, 400, 272
    from oracle import fpformats as F
    h = g.integers(-2, 3, (t, top, inner)).astype(np.float64)
    d = g.integers(-2, 3, (e, hidden, inner)).astype(np.float64)
    ids, _ = choices(t, top, e, seed=9)
    hs = 2.0 ** g.integers(-1, 2, (O.blocks(inner), t * top)).astype(np.float64)
    ds = 2.0 ** g.integers(-1, 2, (e, O.blocks(hidden), O.blocks(inner))).astype(np.float64)
    hq, dq = F.fp32_to_e4m3_code(h), F.fp32_to_e4m3_code(d)
    w = M.ExpertWeights(torch.zeros(e, 2, inner, hidden, dtype=torch.uint8).cuda(),
                        torch.zeros(e, 2, O.blocks(inner), O.blocks(hidden)).cuda(), dev(dq), dev(ds.astype(np.float32)))
    y = M.experts_down(dev(hq), dev(hs.astype(np.float32)), dev(ids), dev((ids >= 0).astype(np.float32)), w)
    values = O.values_rows(hq.reshape(t * top, inner), hs).reshape(t, top, inner)
    want = torch.zeros(t, hidden)
    for i in range(t):
        for j in range(top):
            if ids[i, j] >= 0:
                part = values[i, j] @ O.values_weight(dq[ids[i, j]], ds[ids[i, j]]).T
                want[i] += torch.from_numpy(part).to(torch.bfloat16).float()
    assert torch.equal(y.cpu(), want.to(torch.bfloat16))


def test_the_same_expert_twice_and_ids_out_of_range():
    t, top, e, hidden, inner = 40, 4, 6, 256, 144
    w = M.ExpertWeights(*map(dev, U.expert_weights(e, inner, hidden, seed=1)))
    x = U.activations(t, hidden, seed=2).cuda()
    ids = torch.full((t, top), 3, dtype=torch.int32, device="cuda")
    ids[:, 2] = 1
    weights = torch.full((t, top), 0.25, device="cuda")
    y = M.experts(x, ids, weights, w)
    apart = torch.zeros(t, hidden, device="cuda")
    h, hs = M.experts_up(x, ids, w)
    for j in range(top):
        one = torch.zeros_like(weights)
        one[:, j] = 1.0
        apart += 0.25 * M.experts_down(h, hs, ids, one, w).float()
    assert torch.equal(y, apart.to(torch.bfloat16))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids[7, 1], ids[9, 3], ids[11, 0] = e, 1 << 30, -(1 << 31)
    bad = M.experts(x, ids, weights, w, status=status)
    gone = ids.clone()
    gone[(gone < 0) | (gone >= e)] = -1
    assert int(status) == -1 and torch.equal(bad, M.experts(x, gone, weights, w))


def test_no_tokens():
    w = M.ExpertWeights(*map(dev, U.expert_weights(2, 16, 32, seed=1)))
    x = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    ids, weights = M.route(torch.empty(0, 2, device="cuda"), 1)
    assert M.experts(x, ids, weights, w).shape == (0, 32)
