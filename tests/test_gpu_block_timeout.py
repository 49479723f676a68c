"""Waits inside the products in 8-bit blocks that run out (the test hook has them expect too many bytes): the status word says so,
what was not computed is NaN, and the next call is right."""
import numpy as np
import pytest
import torch

import precision_gemm_token_gb300 as E
from precision_gemm_token_gb300 import blocks as B
from precision_gemm_token_gb300 import moe as M
from tests import moe_util as U

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run_out(call):
    """What `call(status)` gives where its waits run out; before and after that it is right."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = [t.clone() for t in call(status)]
    torch.cuda.synchronize()
    assert int(status) == 0
    E.epilora_test_late_block_copies(True)
    try:
        got = call(status)
        torch.cuda.synchronize()
    finally:
        E.epilora_test_late_block_copies(False)
    assert int(status) == E.EPILORA_ERR_TIMEOUT
    status.zero_()
    again = call(status)
    assert int(status) == 0 and all(torch.equal(a, b) for a, b in zip(again, want))
    return got


# one block, narrow and wide tiles, several tiles a thread block, K over a cluster (whole and cut short)
@pytest.mark.parametrize("m,n,k", [(5, 100, 128), (64, 640, 512), (2000, 40000, 256), (300, 1000, 2064), (32, 4096, 4096),
                                   (3, 130, 9008)])
def test_products(m, n, k):
    x = U.activations(m, k, seed=m).cuda()
    w = B.quantize_weight(U.activations(n, k, seed=n).cuda())
    assert run_out(lambda st: [B.block_linear(x, w, status=st)])[0].isnan().all()


@pytest.mark.parametrize("t,top,e", [(9, 2, 16), (300, 2, 3)])        # few rows an expert, and many
def test_experts(t, top, e):
    w = M.ExpertWeights(*map(dev, U.expert_weights(e, 208, 272, seed=1)))
    x = U.activations(t, 272, seed=t).cuda()
    ids = torch.arange(t * top, dtype=torch.int32, device="cuda").view(t, top) % e
    weights = torch.rand(t, top, device="cuda") + 0.5
    codes, _ = run_out(lambda st: M.experts_up(x, ids, w, status=st))
    assert (codes.view(torch.uint8) & 0x7F == 0x7F).all()                # NaN
    up = M.experts_up(x, ids, w)
    for parts in (torch.bfloat16, torch.float32):
        assert run_out(lambda st: [M.experts_down(*up, ids, weights, w, status=st, parts=parts)])[0].isnan().all()
    assert run_out(lambda st: [M.experts(x, ids, weights, w, status=st)])[0].isnan().all()
