"""The operators in 8-bit blocks on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import fpformats as F
from oracle import moe_oracle as O
from precision_gemm_token_gb300 import blocks as B
from tests import moe_util as U

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("m,k", [(1, 16), (1, 4096), (2, 128), (3, 144), (17, 2064), (64, 7168), (129, 1040), (1000, 272),
                                 (700, 14336)])
def test_block_quant(m, k):
    x = U.activations(m, k, seed=m + k)
    x[m // 2, : min(k, 128)] = 0
    codes, scale = B.block_quant(x.cuda())
    want_c, want_s = O.quant_rows(x.float().numpy())
    assert np.array_equal(scale.cpu().numpy(), want_s)
    assert np.array_equal(F.e4m3_decode(codes.cpu().numpy()), F.e4m3_decode(want_c))


def test_block_quant_strides_and_extremes():
    wide = torch.zeros(40, 3, 512, dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(5)
    wide[:] = torch.randn(40, 3, 512, generator=g)
    wide[0, 1] *= 2.0 ** -120
    wide[1, 1] *= 2.0 ** 100
    wide[2, 1, :] = torch.finfo(torch.bfloat16).max
    wide[3, 1, :] = torch.finfo(torch.bfloat16).tiny
    wide[4, 1, 7::2] = 2.0 ** -133                    # subnormal beside ordinary ones
    x = wide.cuda()[:, 1, :]
    codes, scale = B.block_quant(x)
    want_c, want_s = O.quant_rows(x.float().cpu().numpy())
    assert np.array_equal(scale.cpu().numpy(), want_s)
    assert np.array_equal(F.e4m3_decode(codes.cpu().numpy()), F.e4m3_decode(want_c))


def test_block_quant_nan_and_infinity():
    x = torch.ones(3, 256, dtype=torch.bfloat16)
    x[0, 5], x[1, 130], x[2, 0] = float("nan"), float("inf"), float("-inf")
    codes, scale = B.block_quant(x.cuda())
    v, s = F.e4m3_decode(codes.cpu().numpy()), scale.cpu().numpy()
    one = np.float32(1) / np.float32(448)
    assert s[0, 0] == one and s[1, 0] == one and np.isnan(v[0, 5]) and (np.delete(v[0], 5) == 448).all()
    assert s[0, 1] == one and np.isinf(s[1, 1]) and np.isnan(v[1, 130]) and (np.delete(v[1, 128:], 2) == 0).all()
    assert np.isinf(s[0, 2]) and np.isnan(v[2, 0]) and (v[2, 1:128] == 0).all() and (v[2, 128:] == 448).all()


@pytest.mark.parametrize("n,k", [(1, 16), (128, 128), (130, 144), (257, 1040), (1000, 2064)])
def test_quantize_weight(n, k):
    W = U.activations(n, k, seed=n)
    w = B.quantize_weight(W.cuda())
    codes, scale = O.quant_weight(W.float().numpy())
    assert np.array_equal(w.scale.cpu().numpy(), scale)
    assert np.array_equal(F.e4m3_decode(w.codes.cpu().numpy()), F.e4m3_decode(codes))


SHAPES = [(1, 1, 16), (1, 4096, 128), (1, 6144, 4096), (2, 17, 144), (5, 1000, 2064), (32, 4096, 1024), (33, 129, 272),
          (64, 640, 512), (127, 255, 4096), (128, 128, 128), (129, 257, 1040), (300, 1000, 2064), (512, 2048, 640),
          (1000, 70, 384), (40, 20000, 256), (2000, 4096, 256)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_block_matmul_integers(m, n, k):
    """Small whole numbers and scales that are powers of two: every sum is exact, so is the answer."""
    g = np.random.default_rng(m + n + k)
    a, w = g.integers(-4, 5, (m, k)).astype(np.float64), g.integers(-4, 5, (n, k)).astype(np.float64)
    sa = 2.0 ** g.integers(-1, 2, (O.blocks(k), m))
    sw = 2.0 ** g.integers(-1, 2, (O.blocks(n), O.blocks(k)))
    aq, wq = F.fp32_to_e4m3_code(a), F.fp32_to_e4m3_code(w)
    want = O.values_rows(aq, sa) @ O.values_weight(wq, sw).T
    y = B.block_matmul(dev(aq), dev(sa.astype(np.float32)), B.BlockWeight(dev(wq), dev(sw.astype(np.float32))))
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(torch.bfloat16))


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_block_linear(m, n, k):
    x = U.activations(m, k, seed=3 * m + n)
    codes, scale = U.weight(n, k, seed=k)
    y = B.block_linear(x.cuda(), B.BlockWeight(dev(codes), dev(scale)))
    want, size = O.product(O.values_rows(*O.quant_rows(x.float().numpy())), O.values_weight(codes, scale))
    off = U.sum_bound(k, size)
    U.close(U.f64(y), want, off + U.BF16 * (np.abs(want) + off))


@pytest.mark.parametrize("pad,at", [(0, 0), (1, 0), (3, 1), (16, 0), (16, 8), (40, 5)])
def test_output_of_any_stride_and_alignment(pad, at):
    m, n, k = 131, 333, 272
    x, (codes, scale) = U.activations(m, k, seed=1).cuda(), U.weight(n, k, seed=2)
    w = B.BlockWeight(dev(codes), dev(scale))
    buf = torch.full((m, n + pad + at), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, at:at + n]
    assert B.block_linear(x, w, out=out) is out
    assert torch.equal(out, B.block_linear(x, w))
    assert (buf[:, :at] == 7).all() and (buf[:, at + n:] == 7).all()


def test_strided_input():
    wide = U.activations(50, 3 * 400, seed=9).cuda()
    codes, scale = U.weight(200, 400, seed=4)
    w = B.BlockWeight(dev(codes), dev(scale))
    for i in range(3):
        x = wide[:, 400 * i:400 * (i + 1)]
        assert torch.equal(B.block_linear(x, w), B.block_linear(x.contiguous(), w))


def test_a_row_of_nan_stays_alone():
    x = U.activations(140, 512, seed=8)
    codes, scale = U.weight(300, 512, seed=4)
    w = B.BlockWeight(dev(codes), dev(scale))
    clean = B.block_linear(x.cuda(), w)
    x[7, 3], x[131, 500] = float("nan"), float("inf")
    y = B.block_linear(x.cuda(), w)
    keep = [i for i in range(140) if i not in (7, 131)]
    assert torch.equal(y[keep], clean[keep]) and y[7].isnan().all() and y[131].isnan().all()


def test_no_rows():
    codes, scale = U.weight(300, 512, seed=4)
    w = B.BlockWeight(dev(codes), dev(scale))
    assert B.block_linear(torch.empty(0, 512, dtype=torch.bfloat16, device="cuda"), w).shape == (0, 300)
    q, s = B.block_quant(torch.empty(0, 512, dtype=torch.bfloat16, device="cuda"))
    assert B.block_matmul(q, s, w).shape == (0, 300)
