"""A rotation table without a row, or without an element: refused, where
there is a token to rotate."""
import pytest
import torch

import precision_gemm_token_gb300 as E
from precision_gemm_token_gb300 import attention as A

from .attention_util import Batch, ensure_lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(0, 64), (40, 0), (0, 0)])
def test_empty_table(shape):
    ensure_lib()
    b = Batch([(2, 20)], 4, 2, 64)
    x = torch.ones(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    start, length, table = b.dev("q_start", "kv_len", "table")
    before = b.cache.k.clone()
    with pytest.raises(E.EpiloraError, match="cos_sin: "):
        A.kv_append(x[:, :4], x[:, 4:6], x[:, 6:], b.cache, start, length, table, torch.zeros(shape, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(b.cache.k.view(torch.int16), before.view(torch.int16))
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = A.kv_append(x[:0, :4], x[:0, 4:6], x[:0, 6:], b.cache, start, length, table, torch.zeros(0, 64, device="cuda"))
    assert q.shape == (0, 4, 64)
