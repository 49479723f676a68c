"""The largest sizes of the operators in 8-bit blocks: beyond them a sum of a size and a tile's would not fit 32 bits, so
they are refused before anything is enqueued (fake addresses, only where no device exists to launch on)."""
import pytest
import torch

import precision_gemm_token_gb300 as E

FAKE = 0x10000
BIG, UNSUP = E.BLOCK_MAX_SIZE, E.EPILORA_ERR_UNSUPPORTED
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only where nothing can launch")
# just beyond, and the last one of 32 bits (of those that are multiples of 16)
ROWS, WIDTHS = (BIG + 1, 2 ** 31 - 128, 2 ** 31 - 1), (BIG + 16, 2 ** 31 - 16)


@pytest.fixture(scope="module", autouse=True)
def lib():
    E.build()
    return E.load()


def test_the_limit_is_the_headers():
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "include", "epilora.h")
    assert int(re.search(r"define EPILORA_BLOCK_MAX_SIZE (\w+)", open(path).read()).group(1), 0) == BIG


@no_gpu
def test_rows_and_columns():
    for m in ROWS:
        assert E.epilora_block_quant(FAKE, m, 16, 16, FAKE, FAKE, m, 0) == UNSUP
        assert E.epilora_block_quant_weight(FAKE, m, 16, 16, FAKE, FAKE, 0) == UNSUP
        assert E.epilora_block_matmul(m, 1, 16, FAKE, FAKE, m, FAKE, FAKE, FAKE, 1, None, 0) == UNSUP
        assert E.epilora_block_matmul(1, m, 16, FAKE, FAKE, 1, FAKE, FAKE, FAKE, m, None, 0) == UNSUP
        assert E.epilora_block_linear_workspace_bytes(m, 16) == 0
        for size in ((m, 1), (1, m)):
            assert E.epilora_block_linear(*size, 16, FAKE, 16, FAKE, FAKE, FAKE, size[1], FAKE, 1 << 60, None, 0) == UNSUP


@no_gpu
def test_widths():
    for k in WIDTHS:
        assert E.epilora_block_quant(FAKE, 1, k, k, FAKE, FAKE, 1, 0) == UNSUP
        assert E.epilora_block_quant_weight(FAKE, 1, k, k, FAKE, FAKE, 0) == UNSUP
        assert E.epilora_block_matmul(1, 1, k, FAKE, FAKE, 1, FAKE, FAKE, FAKE, 1, None, 0) == UNSUP
        assert E.epilora_block_linear(1, 1, k, FAKE, k, FAKE, FAKE, FAKE, 1, FAKE, 1 << 60, None, 0) == UNSUP
        assert E.epilora_block_linear_workspace_bytes(1, k) == 0
        for size in ((k, 16), (16, k)):
            assert E.epilora_moe_workspace_bytes(E.MOE_UP | E.MOE_DOWN, 1, 1, 1, *size) == 0
            up = E.epilora_moe_experts_up(1, 1, 1, *size, FAKE, size[0], FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 60, None, 0)
            assert up == UNSUP
            for down in (E.epilora_moe_experts_down, E.epilora_moe_experts_down_f32):
                assert down(1, 1, 1, *size, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, size[0], FAKE, 1 << 60, None, 0) == UNSUP


def test_the_largest_sizes_have_a_workspace():
    assert E.epilora_block_linear_workspace_bytes(BIG, 16) >= BIG * 16
    assert E.epilora_block_linear_workspace_bytes(1, BIG) >= BIG
