"""How the calls in 8-bit blocks and of the mixture of experts are made: streams, captured graphs, shared workspaces,
skewed and padded batches, sizes past 32 bits, refusals on GPU tensors."""
import numpy as np
import pytest
import torch

import precision_gemm_token_gb300 as E
from oracle import moe_oracle as O
from precision_gemm_token_gb300 import blocks as B
from precision_gemm_token_gb300 import moe as M
from tests import moe_util as U

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def block_weight(n, k, seed):
    return B.BlockWeight(*map(dev, U.weight(n, k, seed)))


def experts_of(e, inner, hidden, seed=1):
    return M.ExpertWeights(*map(dev, U.expert_weights(e, inner, hidden, seed)))


# few rows with K over 2, 4 and 8 thread blocks, whole and cut short
@pytest.mark.parametrize("m,n,k", [(1, 6144, 4096), (32, 4096, 4096), (5, 1000, 8192), (32, 2000, 16384), (17, 130, 12000),
                                   (1, 1, 16384), (31, 2400, 9008)])
def test_few_rows_over_a_cluster(m, n, k):
    x = U.activations(m, k, seed=m)
    codes, scale = U.weight(min(n, 512), k, seed=k)
    codes, scale = np.tile(codes, (-(-n // 512) or 1, 1))[:n], np.tile(scale, (-(-n // 512) or 1, 1))[:O.blocks(n)]
    y = B.block_linear(x.cuda(), B.BlockWeight(dev(codes), dev(scale)))
    want, size = O.product(O.values_rows(*O.quant_rows(x.float().numpy())), O.values_weight(codes, scale))
    off = U.sum_bound(k, size)
    U.close(U.f64(y), want, off + U.BF16 * (np.abs(want) + off))


# tiles of every width (and the product turned round), rows of the output that start anywhere
@pytest.mark.parametrize("m,n,k", [(2000, 4097, 256), (300, 6001, 144), (150, 2003, 1040), (64, 501, 4096), (3000, 23, 576),
                                   (9, 1999, 4096), (257, 20001, 128)])
def test_odd_widths(m, n, k):
    w = block_weight(n, k, n)
    x = U.activations(m, k, seed=m).cuda()
    room = torch.zeros(m, -(-n // 16) * 16, dtype=torch.bfloat16, device="cuda")
    want = B.block_linear(x, w, out=room[:, :n])
    assert torch.equal(B.block_linear(x, w), want)
    odd = torch.full((m, n + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    B.block_linear(x, w, out=odd[:, 1:n + 1])
    assert torch.equal(odd[:, 1:n + 1], want) and (odd[:, 0] == 7).all() and (odd[:, n + 1:] == 7).all()
    assert (room[:, n:] == 0).all()
    rows = [0, m // 2, m - 1]
    exact, size = O.product(O.values_rows(*O.quant_rows(x[rows].float().cpu().numpy())),
                            O.values_weight(w.codes.cpu().numpy(), w.scale.cpu().numpy()))
    off = U.sum_bound(k, size)
    U.close(U.f64(want[rows]), exact, off + U.BF16 * (np.abs(exact) + off))


@pytest.mark.parametrize("t,e", [(100, 64), (300, 64), (40, 128)])
def test_everybody_at_one_expert(t, e):
    """Batches that are few rows an expert on average, all of them with one."""
    w = experts_of(4, 208, 272)
    wide = M.ExpertWeights(*(torch.cat([p.roll(1, 0)] * (e // 4)) for p in (w.gate_up, w.gate_up_scale, w.down, w.down_scale)))
    x = U.activations(t, 272, seed=t).cuda()
    ids = torch.full((t, 1), 6, dtype=torch.int32, device="cuda")            # the same weights as expert 1 of w
    weights = torch.rand(t, 1, device="cuda")
    codes, scale = M.experts_up(x, ids, wide)
    h, bound = U.up_expected(*O.quant_rows(x.float().cpu().numpy()), ids.cpu().numpy() - 5, w.gate_up.cpu().numpy(),
                             w.gate_up_scale.cpu().numpy())
    U.check_quantized(codes, scale, h, bound)
    y = M.experts_down(codes, scale, ids, weights, wide)
    want, off = U.down_expected(codes.cpu().numpy().reshape(t, -1), scale.cpu().numpy(), ids.cpu().numpy() - 5,
                                weights.cpu().numpy(), w.down.cpu().numpy(), w.down_scale.cpu().numpy())
    U.close(U.f64(y), want, off)


@pytest.mark.parametrize("t,top,e", [(1, 1, 1024), (50, 8, 1000), (3000, 6, 512), (40, 32, 64), (7, 17, 33)])
def test_many_experts(t, top, e):
    g = np.random.default_rng(t)
    ids = np.argsort(g.random((t, e)), 1)[:, :top].astype(np.int32)
    w = experts_of(3, 32, 48)
    wide = M.ExpertWeights(*(p[torch.arange(e, device="cuda") % 3].contiguous()
                             for p in (w.gate_up, w.gate_up_scale, w.down, w.down_scale)))
    x, weights = U.activations(t, 48, seed=1).cuda(), dev(g.random((t, top)).astype(np.float32))
    a = M.experts_up(x, dev(ids), wide)
    b = M.experts_up(x, dev(ids % 3), w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(M.experts_down(*a, dev(ids), weights, wide), M.experts_down(*b, dev(ids % 3), weights, w))


def test_results_repeat_bit_for_bit():
    w = experts_of(16, 384, 640)
    x = U.activations(700, 640, seed=2).cuda()
    ids, weights = M.route(torch.randn(700, 16, device="cuda"), 4)
    ws = B.BlockWorkspace("cuda")
    y = M.experts(x, ids, weights, w, workspace=ws)
    for _ in range(5):
        assert torch.equal(M.experts(x, ids, weights, w, workspace=ws), y)


def layer(x, router, w, dense, ws, **kw):
    """What a mixture layer calls: a router's logits, the choice, the experts, and a dense projection beside them."""
    logits = B.block_linear(x, router, workspace=ws, **kw)
    ids, weights = M.route(logits, 3, scoring="sigmoid", groups=4, top_groups=2, group_best=2, **kw)
    y = M.experts(x, ids, weights, w, workspace=ws, **kw)
    return ids, weights, y, B.block_linear(y, dense, workspace=ws, **kw)


def parts(tokens, seed=3):
    return (U.activations(tokens, 256, seed).cuda(), block_weight(16, 256, 1), experts_of(16, 144, 256),
            block_weight(300, 256, 2))


@pytest.mark.parametrize("tokens", [1, 20, 500])
def test_a_captured_layer_follows_its_input(tokens):
    x, *w = parts(tokens)
    ws = B.BlockWorkspace("cuda")
    layer(x, *w, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(x, *w, ws)
    for seed in (5, 6):
        x.copy_(U.activations(tokens, 256, seed))
        g.replay()
        want = layer(x, *w, B.BlockWorkspace("cuda"))
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_graphs_and_eager_calls_share_a_workspace_that_grows():
    ws = B.BlockWorkspace("cuda")
    small, large = parts(8), parts(600, seed=9)
    graphs = []
    for p in (small, large):          # (the first graph's buffer has to outlive the growth for the second)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer(*p, ws)
        graphs.append((g, out, p))
    huge = parts(3000, seed=4)
    layer(*huge, ws)
    filler = [torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(2):
        for g, out, p in graphs:
            g.replay()
            layer(*huge, ws)
            want = layer(*p, B.BlockWorkspace("cuda"))
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    del filler


def test_another_stream():
    x, *w = parts(64)
    want = layer(x, *w, B.BlockWorkspace("cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = B.BlockWorkspace("cuda")
    got = layer(x, *w, ws, stream=side)
    handle = torch.cuda.Stream()
    handle.wait_stream(torch.cuda.current_stream())
    raw = layer(x, *w, None, stream=handle.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.current_stream().wait_stream(handle)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(raw, want))


def test_a_weight_that_the_kernel_before_writes():
    """No call reads a weight before the kernel that quantizes it has finished."""
    W = [U.activations(2048, 1024, seed=s).cuda() for s in (1, 2)]
    x = U.activations(16, 1024, seed=3).cuda()
    ws = B.BlockWorkspace("cuda")
    codes, scale = B.block_quant(x)
    for make in (lambda w: B.block_linear(x, w, workspace=ws), lambda w: B.block_matmul(codes, scale, w)):
        want = [make(B.quantize_weight(m)) for m in W]
        for _ in range(4):
            for m, y in zip(W, want):
                assert torch.equal(make(B.quantize_weight(m)), y)


def test_offsets_past_32_bits():
    m, k = 150000, 16384                                # 2.46e9 elements
    base = U.activations(8, k, seed=1).cuda()
    x = base.repeat(m // 8, 1)
    codes, scale = B.block_quant(x)
    want_c, want_s = B.block_quant(base)
    assert torch.equal(codes.view(-1, 8, k)[[0, -1]], want_c.expand(2, 8, k))
    assert torch.equal(scale[:, -8:], want_s) and torch.equal(scale[:, :8], want_s)
    del x
    w = block_weight(130, k, 2)
    y = B.block_matmul(codes, scale, w)
    assert torch.equal(y.view(-1, 8, 130)[-1], y[:8]) and torch.equal(y[-8:], y[:8])
    want, size = O.product(O.values_rows(want_c.cpu().numpy(), want_s.cpu().numpy()),
                           O.values_weight(w.codes.cpu().numpy(), w.scale.cpu().numpy()))
    off = U.sum_bound(k, size)
    U.close(U.f64(y[-8:]), want, off + U.BF16 * (np.abs(want) + off))


def test_weights_past_32_bits():
    e, inner, hidden = 40, 4096, 8192                   # 2.7e9 codes of gate and up, 1.3e9 of down
    one = U.expert_weights(1, inner, hidden, seed=1)
    small = M.ExpertWeights(*map(dev, one))
    wide = M.ExpertWeights(*(p.expand(e, *p.shape[1:]).contiguous()
                             for p in (small.gate_up, small.gate_up_scale, small.down, small.down_scale)))
    x = U.activations(4, hidden, seed=1).cuda()
    ids = torch.tensor([[39, 1], [38, 39], [0, 20], [39, 39]], dtype=torch.int32, device="cuda")
    weights = torch.rand(4, 2, device="cuda")
    for t in (1, 40):                                   # (few rows an expert, then many)
        xs, i, f = x.repeat(t, 1), ids.repeat(t, 1), weights.repeat(t, 1)
        a, b = M.experts_up(xs, i, wide), M.experts_up(xs, torch.zeros_like(i), small)
        if t == 40:
            assert torch.equal(a[0][:4], a[0][-4:])
        h, bound = U.up_expected(*O.quant_rows(x.float().cpu().numpy()), np.zeros((4, 2), np.int32), one[0], one[1])
        for c, s in (a, b):
            U.check_quantized(c[-4:], s.view(-1, 4 * t, 2)[:, -4:].reshape(s.shape[0], -1), h, bound)
        y = M.experts_down(*a, i, f, wide)
        want, off = U.down_expected(a[0][-4:].cpu().numpy().reshape(8, -1),
                                    a[1].view(-1, 4 * t, 2)[:, -4:].reshape(a[1].shape[0], -1).cpu().numpy(),
                                    np.zeros((4, 2), np.int32), weights.cpu().numpy(), one[2], one[3])
        U.close(U.f64(y[-4:]), want, off)


def test_refusals():
    x, router, w, dense = parts(6)
    ids, weights = M.route(torch.randn(6, 16, device="cuda"), 2)
    h, hs = M.experts_up(x, ids, w)
    ws = B.BlockWorkspace("cuda")
    bad = [
        lambda: B.block_quant(x.float()), lambda: B.block_quant(x[:, 1:]), lambda: B.block_quant(x[0]),
        lambda: B.block_quant(x.T), lambda: B.block_quant(x[:, :24]),
        lambda: B.block_quant(x, scale=torch.empty(6, 2, device="cuda")),
        lambda: B.block_linear(x[:, :128], dense), lambda: B.block_linear(x, dense, out=torch.empty(6, 300, device="cuda")),
        lambda: B.block_linear(x, dense, out=torch.empty(5, 300, dtype=torch.bfloat16, device="cuda")),
        lambda: B.block_matmul(h, hs, dense), lambda: B.block_matmul(*B.block_quant(x)[::-1], dense),
        lambda: B.block_linear(x, dense, status=torch.zeros(1, device="cuda")),
        lambda: M.route(torch.zeros(4, 8, dtype=torch.float16, device="cuda"), 2),
        lambda: M.route(torch.zeros(4, 8, device="cuda"), 0), lambda: M.route(torch.zeros(4, 8, device="cuda"), 9),
        lambda: M.route(torch.zeros(4, 8, device="cuda"), 2, scoring="relu"),
        lambda: M.route(torch.zeros(4, 8, device="cuda"), 2, bias=torch.zeros(7, device="cuda")),
        lambda: M.route(torch.zeros(4, 8, device="cuda"), 2, groups=3),
        lambda: M.experts_up(x, ids[:5], w), lambda: M.experts_up(x, ids.long(), w), lambda: M.experts_up(x[:, :128], ids, w),
        lambda: M.experts_down(h, hs, ids, weights.double(), w), lambda: M.experts_down(h[:, :1], hs, ids, weights, w),
        lambda: M.experts_down(h, hs[:, :6], ids, weights, w), lambda: M.experts(x, ids, weights[:, :1], w, workspace=ws),
        lambda: M.experts(x, ids.T.contiguous().T, weights, w, workspace=ws)]
    for i, call in enumerate(bad):
        with pytest.raises(E.EpiloraError):
            call()
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()
