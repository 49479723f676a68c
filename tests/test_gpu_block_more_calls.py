"""Calls in 8-bit blocks that the header allows and the helpers do not make (scales with a stride, rows of a larger batch),
and batches at their edges: NaN in weights and in tokens, nobody routed anywhere, two streams at once."""
import numpy as np
import pytest
import torch

import precision_gemm_token_gb300 as E
from oracle import moe_oracle as O
from precision_gemm_token_gb300 import blocks as B
from precision_gemm_token_gb300 import moe as M
from tests import moe_util as U

pytestmark = pytest.mark.gpu
NAN = 0x7F                      # E4M3


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def block_weight(n, k, seed):
    return B.BlockWeight(*map(dev, U.weight(n, k, seed)))


def experts_of(e, inner, hidden, seed=1):
    return M.ExpertWeights(*map(dev, U.expert_weights(e, inner, hidden, seed)))


# narrow, wide, K over a cluster
SHAPES = [(40, 300, 272), (700, 30000, 256), (20, 640, 4096)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_scales_with_a_stride_and_rows_of_a_larger_batch(m, n, k):
    x, w = U.activations(m, k, seed=m).cuda(), block_weight(n, k, 3)
    nb, ld = -(-k // 128), m + 13
    codes = torch.zeros(m, k, dtype=torch.uint8, device="cuda")
    scale = torch.full((nb, ld), float("nan"), device="cuda")
    assert E.epilora_block_quant(x, m, k, k, codes, scale, ld) == E.EPILORA_OK
    want_codes, want_scale = B.block_quant(x)
    assert torch.equal(codes, want_codes) and torch.equal(scale[:, :m], want_scale) and scale[:, m:].isnan().all()
    want = B.block_matmul(want_codes, want_scale, w)
    exact, size = O.product(O.values_rows(codes.cpu().numpy(), want_scale.cpu().numpy()),
                            O.values_weight(w.codes.cpu().numpy(), w.scale.cpu().numpy()))
    off = U.sum_bound(k, size)
    for first, rows in ((0, m), (m // 3, m - m // 3), (m - 1, 1)):
        y = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
        rc = E.epilora_block_matmul(rows, n, k, codes[first:], scale[0, first:], ld, w.codes, w.scale, y, n)
        assert rc == E.EPILORA_OK and (rows < m or torch.equal(y, want))
        part = np.s_[first:first + rows]                # (fewer rows may be summed in another order)
        U.close(U.f64(y), exact[part], off[part] + U.BF16 * (np.abs(exact[part]) + off[part]))


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_nan_in_a_weight_stays_in_its_column(m, n, k):
    x, (codes, scale) = U.activations(m, k, seed=m).cuda(), map(dev, U.weight(n, k, 3))
    want = B.block_linear(x, B.BlockWeight(codes, scale))
    bad = [0, n // 2, n - 1]
    codes[bad, k - 1] = NAN
    y = B.block_linear(x, B.BlockWeight(codes, scale))
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert y[:, bad].isnan().all() and torch.equal(y[:, keep], want[:, keep])


@pytest.mark.parametrize("t,top,e", [(20, 2, 12), (300, 2, 4)])          # few rows an expert, and many
def test_nan_in_experts(t, top, e):
    hidden, inner = 272, 208
    w = experts_of(e, inner, hidden)
    x = U.activations(t, hidden, seed=t).cuda()
    ids = torch.arange(t * top, dtype=torch.int32, device="cuda").view(t, top) % e
    weights = torch.rand(t, top, device="cuda") + 0.5
    codes, scale = M.experts_up(x, ids, w)
    for parts in (torch.bfloat16, torch.float32):
        want = M.experts(x, ids, weights, w, parts=parts)
        # a token
        sick = x.clone()
        sick[t // 2, 5] = float("nan")
        y = M.experts(sick, ids, weights, w, parts=parts)
        rest = [i for i in range(t) if i != t // 2]
        assert y[t // 2].isnan().all() and torch.equal(y[rest], want[rest])
        # a column of one expert's down weights
        d = w.down.clone()
        d[1, 7, 3] = NAN
        y = M.experts_down(codes, scale, ids, weights, M.ExpertWeights(w.gate_up, w.gate_up_scale, d, w.down_scale),
                           parts=parts)
        hit = (ids == 1).any(1)
        clean = M.experts_down(codes, scale, ids, weights, w, parts=parts)
        assert y[hit, 7].isnan().all() and torch.equal(y[~hit], clean[~hit])
        assert torch.equal(torch.cat([y[:, :7], y[:, 8:]], 1), torch.cat([clean[:, :7], clean[:, 8:]], 1))
    # a row of one expert's gate: one element of the inner rows, whose block keeps the scale of the others
    gu = w.gate_up.clone()
    gu[1, 0, 9, 3] = NAN
    got, got_scale = M.experts_up(x, ids, M.ExpertWeights(gu, w.gate_up_scale, w.down, w.down_scale))
    hit = ids == 1
    assert ((got[hit][:, 9] & 0x7F) == NAN).all() and torch.equal(got[~hit], codes[~hit])
    assert torch.equal(got[..., 128:], codes[..., 128:]) and torch.equal(got_scale[1], scale[1])


@pytest.mark.parametrize("t", [1, 50, 600])
def test_nobody_is_routed_anywhere(t):
    w = experts_of(4, 144, 256)
    x, ids = U.activations(t, 256, 1).cuda(), torch.full((t, 3), -1, dtype=torch.int32, device="cuda")
    weights = torch.full((t, 3), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scale = M.experts_up(x, ids, w, status=status)
    assert (codes == 0).all() and (scale == 0).all()
    for parts in (torch.bfloat16, torch.float32):
        assert (M.experts_down(codes, scale, ids, weights, w, status=status, parts=parts) == 0).all()
        assert (M.experts(x, ids, weights, w, status=status, parts=parts) == 0).all()
    assert int(status) == 0


def test_two_streams_at_once():
    w, dense = experts_of(8, 208, 272), block_weight(500, 272, 2)
    sets = [(U.activations(t, 272, t).cuda(), torch.randn(t, 8, device="cuda"), B.BlockWorkspace("cuda")) for t in (70, 900)]

    def layer(x, logits, ws):
        ids, weights = M.route(logits, 2)
        return M.experts(x, ids, weights, w, workspace=ws), B.block_linear(x, dense, workspace=ws)
    want = [layer(x, l, B.BlockWorkspace("cuda")) for x, l, _ in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(*sets[i]))
    torch.cuda.synchronize()
    for i, runs in enumerate(got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))
