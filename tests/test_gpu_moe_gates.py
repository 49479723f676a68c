"""Gated products at the ends of the activation: gates where the exponential leaves 32 bits, beside large up values."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from precision_gemm_token_gb300 import moe as M
from tests import moe_util as U

pytestmark = pytest.mark.gpu
GATES = [-1000.0, -104.0, -90.0, -88.8, -88.0, -87.5, -87.2, -86.0, -60.0, -17.0, -1.0, -1e-20, 0.0, 1e-20, 1.0, 17.0, 60.0,
         89.0, 1000.0]


@pytest.mark.parametrize("t", [1, 40])          # few rows an expert, and many
@pytest.mark.parametrize("up", [1.0, 1e30, -1e30])
def test_gates(t, up):
    """Expert e's gates are GATES[e] in every column, its up values `up`, within the rounding of the scales."""
    n, hidden, inner = len(GATES), 16, 144
    one = 0x38                                   # E4M3 of 1
    codes = np.full((n, 2, inner, hidden), one, np.uint8)
    scale = np.zeros((n, 2, O.blocks(inner), 1), np.float32)
    for e, g in enumerate(GATES):
        codes[e, 0] |= 0x80 if g < 0 else 0
        scale[e, 0] = abs(g) / hidden
    codes[:, 1] |= 0x80 if up < 0 else 0
    scale[:, 1] = abs(up) / hidden
    w = M.ExpertWeights(*(torch.from_numpy(a).cuda() for a in (
        codes, scale, np.zeros((n, hidden, inner), np.uint8), np.zeros((n, 1, O.blocks(inner)), np.float32))))
    x = torch.ones(t * n, hidden, dtype=torch.bfloat16)
    ids = (np.arange(t * n, dtype=np.int32) % n)[:, None]
    got, got_scale = M.experts_up(x.cuda(), torch.from_numpy(ids).cuda(), w)
    h, bound = U.up_expected(*O.quant_rows(x.float().numpy()), ids, codes, scale)
    # silu is 0 where it is less than 2^-119; below 2^-126 a 32-bit number, as h in 64 bits is not
    bound += 2.0 ** -119 * abs(up) + 2.0 ** -126
    U.check_quantized(got, got_scale, h, bound)
