"""E4M3 caches where a few positions own a row of the softmax and very many
others, each far below them, hold the rest of its mass together (a long
context behind a few dominant tokens)."""
import math

import numpy as np
import pytest
import torch

import precision_gemm_token_gb300 as E
from oracle import fpformats as F
from precision_gemm_token_gb300 import attention as A

from .attention_util import BF16_U, FP16_U, ensure_lib, f64, lse_bound, status_buf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("gap", [16.0, 22.4, 25.4, 28.0])
def test_dominant_positions_over_a_long_context(dim, n, gap):
    """Positions 0, 32, 64 and 96 score `gap` powers of two above the others
    (one for each of the parts in which a tile's first 128 positions may be
    taken); their values are 0, the others' 1. As many sequences as thread
    blocks share the pages, so that hardly any is cut and the dominant
    positions stand in the same running maximum as the others.

    The bound: the output's rounding and the weights' own as elsewhere; and
    weights below fp16's normal range, whose largest of a row is at least 2^7
    there, are off by at most 2^-25 each, 2^-32 of the largest, so that m
    positions shift the quotient by at most m 2^-32."""
    m, page, group = 1 << 17, 256, 8
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seqs = 2 * sms if n == 1 else sms
    one = int(F.fp32_to_e4m3_code(np.float32([1.0]))[0])
    k = torch.zeros(m // page, 1, page, dim, dtype=torch.uint8)
    v = torch.full_like(k, one)
    for p in (0, 32, 64, 96):
        k[0, 0, p], v[0, 0, p] = one, 0
    k_scale = torch.tensor([gap * math.log(2.0)], dtype=torch.float32)
    cache = A.PagedKVCache(k.cuda(), v.cuda(), k_scale.cuda(), torch.ones(1, device="cuda"))
    q = torch.ones(seqs * n, group, dim, dtype=torch.bfloat16, device="cuda")
    start = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * n
    length = torch.full((seqs,), m, dtype=torch.int32, device="cuda")
    table = torch.arange(m // page, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    lse, st = torch.zeros(seqs * n, group, device="cuda"), status_buf()
    o = A.paged_attention(q, cache, start, length, table, max_new=n, scale=1.0 / dim, lse=lse, status=st)
    assert int(st.item()) == 0
    # token i sees m - n + i + 1 positions; a dominant one scores k_scale, the others 0
    seen = m - n + 1 + np.arange(n)
    top = float(k_scale.double())
    rest = (seen - 4) * math.exp(-top)
    want = rest / (4 + rest)
    bound = BF16_U * want + (FP16_U + 2.0 ** -16 * top + 2.0 ** -14) * want + seen * 2.0 ** -32
    err = np.abs(f64(o).reshape(seqs, n, -1) - want[None, :, None]).max((0, 2))
    assert (err <= bound).all(), (err / bound, err / want)
    want_lse = top + np.log(4 + rest)
    err = np.abs(f64(lse).reshape(seqs, n, -1) - want_lse[None, :, None]).max((0, 2))
    assert (err <= lse_bound(want_lse, top)).all()
