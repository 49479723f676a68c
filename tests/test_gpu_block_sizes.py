"""The largest sizes that the operators in 8-bit blocks take: rows, and columns, up to EPILORA_BLOCK_MAX_SIZE."""
import numpy as np
import pytest
import torch

import precision_gemm_token_gb300 as E
from precision_gemm_token_gb300 import blocks as B
from tests import moe_util as U

pytestmark = pytest.mark.gpu
BIG = E.BLOCK_MAX_SIZE          # a multiple of 65536


def parts(n):
    """Runs of 4096 rows: the first, about the middle, and the last."""
    return [slice(i, i + 4096) for i in (0, n // 2 // 4096 * 4096, n - 4096)]


def test_rows():
    base = U.activations(4096, 16, seed=1).cuda()
    x = base.repeat(BIG // 4096, 1)                     # 69 GB
    codes, scale = B.block_quant(x)
    want, want_scale = B.block_quant(base)
    del x
    w = B.quantize_weight(U.activations(1, 16, seed=2).cuda())
    y = B.block_matmul(codes, scale, w)
    want_y = B.block_matmul(want, want_scale, w)
    for p in parts(BIG):
        assert torch.equal(codes[p], want) and torch.equal(scale[:, p], want_scale) and torch.equal(y[p], want_y)


def test_columns():
    base = U.activations(4096, 16, seed=3).cuda()
    w = B.quantize_weight(base.repeat(BIG // 4096, 1))
    want = B.quantize_weight(base)
    x = U.activations(2, 16, seed=4).cuda()
    y, want_y = B.block_linear(x, w), B.block_linear(x, want)
    for p in parts(BIG):
        blocks = slice(p.start // 128, p.stop // 128)
        assert torch.equal(w.codes[p], want.codes) and torch.equal(w.scale[blocks], want.scale)
        assert torch.equal(y[:, p], want_y)


def test_a_width():
    k = BIG // 16                                       # 134 million: a million blocks of K
    x = torch.zeros(3, k, dtype=torch.bfloat16, device="cuda")
    x[:, :128], x[:, -16:] = 1.0, 2.0
    w = B.quantize_weight(torch.ones(40, k, dtype=torch.bfloat16, device="cuda"))
    y = B.block_linear(x, w)
    exact = np.float64(128 + 32)                        # ones and twos, each 448 times its scale within 2^-24
    assert (np.abs(U.f64(y) - exact) <= exact * (U.BF16 + 2.0 ** -20)).all()
