"""BlockWorkspace that grows: no buffer goes back to the allocator while a stream that it was used on may still have work."""
import pytest
import torch

from precision_gemm_token_gb300 import blocks as B
from tests import moe_util as U

pytestmark = pytest.mark.gpu


def calls():
    w = B.quantize_weight(U.activations(128, 1024, 1).cuda())
    small, large = (U.activations(m, 1024, m).cuda() for m in (500, 5000))        # half a MB, and five
    return w, small, large


def at(ws):
    return ws._buf.data_ptr()


def test_a_raw_handle_beside_the_stream_of_the_buffer():
    w, small, large = calls()
    ws = B.BlockWorkspace("cuda")
    want = B.block_linear(small, w, workspace=ws)
    old, size = at(ws), ws._buf.numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = B.block_linear(small, w, workspace=ws, stream=side.cuda_stream)
    B.block_linear(large, w, workspace=ws, stream=side.cuda_stream)               # grows
    assert at(ws) != old
    # the current stream does not wait for the other one: it must not be given the old buffer
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() != old for t in others)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)


def test_handles_alone_keep_nothing():
    """A buffer made and used on the same handle goes back to that stream's memory, where reuse is in order."""
    w, small, large = calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = B.BlockWorkspace("cuda")
    for x in (small, large):
        B.block_linear(x, w, workspace=ws, stream=side.cuda_stream)
    assert ws._kept == []
    torch.cuda.synchronize()


def test_streams_that_torch_owns_keep_nothing():
    w, small, large = calls()
    side = torch.cuda.Stream()
    ws = B.BlockWorkspace("cuda")
    B.block_linear(small, w, workspace=ws)
    side.wait_stream(torch.cuda.current_stream())
    for x in (small, large):
        B.block_linear(x, w, workspace=ws, stream=side)
    assert ws._kept == []
    torch.cuda.synchronize()
