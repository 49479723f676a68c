"""quantize_experts: each matrix as quantize_weight has it, in the memory of the result alone, on any stream."""
import pytest
import torch

import precision_gemm_token_gb300 as E
from precision_gemm_token_gb300 import blocks as B
from precision_gemm_token_gb300 import moe as M
from tests import moe_util as U

pytestmark = pytest.mark.gpu


def weights(n, inner, hidden, seed=1):
    return tuple(U.activations(n * a, b, seed + i).view(n, a, b).cuda()
                 for i, (a, b) in enumerate(((inner, hidden), (inner, hidden), (hidden, inner))))


def check(w, gate, up, down):
    for e in range(gate.shape[0]):
        for which, m in enumerate((gate[e], up[e], down[e])):
            want = B.quantize_weight(m)
            codes, scale = (w.gate_up[e, which], w.gate_up_scale[e, which]) if which < 2 else (w.down[e], w.down_scale[e])
            assert torch.equal(codes, want.codes) and torch.equal(scale, want.scale)


@pytest.mark.parametrize("n,inner,hidden", [(1, 16, 16), (3, 144, 400), (5, 256, 128), (2, 208, 1040)])
def test_each_matrix(n, inner, hidden):
    parts = weights(n, inner, hidden)
    check(M.quantize_experts(*parts), *parts)
    wide = torch.zeros(n, inner, hidden + 24, dtype=torch.bfloat16, device="cuda")      # rows with a stride of their own
    wide[..., 8:8 + hidden] = parts[0]
    check(M.quantize_experts(wide[..., 8:8 + hidden], *parts[1:]), *parts)


def test_memory():
    n, inner, hidden = 16, 512, 1024
    parts = weights(n, inner, hidden)
    M.quantize_experts(*parts)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    w = M.quantize_experts(*parts)
    made = [w.gate_up, w.gate_up_scale, w.down, w.down_scale]
    # a tensor counts as the block that the allocator gives it: up to 512 bytes more, and in a cached block what is left
    # of it where that is less than 1 MiB (it is not split off then). A second copy of the codes would be 25 MB.
    assert torch.cuda.max_memory_allocated() - before <= sum(t.numel() * t.element_size() + 512 + (1 << 20) for t in made)


def test_another_stream():
    parts = weights(4, 144, 400)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w = M.quantize_experts(*parts, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(w, *parts)


def test_refusals():
    gate, up, down = weights(2, 48, 32)
    for bad in ((gate[0], up[0], down[0]), (gate[:0], up[:0], down[:0]), (gate, up[:1], down), (gate, up, gate),
                (gate.float(), up, down), (gate, up, down.transpose(1, 2).contiguous().transpose(1, 2)),
                (gate.cpu(), up, down), (gate, up.cpu(), down), (gate[:, :40], up[:, :40], down[..., :40])):
        with pytest.raises(E.EpiloraError):
            M.quantize_experts(*bad)
    torch.cuda.synchronize()
