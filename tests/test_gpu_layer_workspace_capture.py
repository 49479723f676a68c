"""A projection's workspace that grows under a graph capture: its zero fill is
the graph's, so every other call has to find the head zeroed by itself."""
import re

import pytest
import torch

import precision_gemm_token_gb300 as E
from precision_gemm_token_gb300 import tensors as T
from synth import make_projection

from .gpu_util import FP8, ensure_lib, status_buf

pytestmark = pytest.mark.gpu


@pytest.fixture
def dirty():
    """A graph memory pool whose free blocks hold ones."""
    ensure_lib()
    pool, g = torch.cuda.graph_pool_handle(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, pool=pool):
        x = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
        del x
    g.replay()
    torch.cuda.synchronize()
    yield pool
    del g


def layer(M=1, K=4096, N=1024):
    p = make_projection(M, K, N, 2, 16, seed=3, device="cuda")
    w = T.quantize_weight(p.W, FP8)
    ref = T.layer_forward(p.X, w, p.A, p.B, p.idx, p.mask)
    torch.cuda.synchronize()
    return (p.X, w, p.A, p.B, p.idx, p.mask), ref


@pytest.mark.parametrize("M", [1, 40])
def test_head_is_zero_before_the_first_replay(dirty, M):
    args, ref = layer(M)
    ws, st, Y = T.LayerWorkspace("cuda"), status_buf(), torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, pool=dirty):
        T.layer_forward(*args, workspace=ws, status=st, Y=Y)
    assert not ws.get(FP8, M, 4096, 16, 1024)[:E.WORKSPACE_SYNC_BYTES].any()
    for _ in range(2):
        assert torch.equal(T.layer_forward(*args, workspace=ws, status=st), ref)
        Y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, ref) and int(st.item()) == 0


def test_prepared_under_capture(dirty):
    args, ref = layer()
    st, Y = status_buf(), torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, pool=dirty):
        call = T.PreparedLayer(*args, workspace=T.LayerWorkspace("cuda"), status=st, Y=Y)
        call()
    for _ in range(2):
        Y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, ref) and int(st.item()) == 0


def test_an_eager_workspace_is_not_zeroed_again():
    """Grown outside a capture it keeps what calls leave in its head."""
    args, ref = layer()
    ws = T.LayerWorkspace("cuda")
    T.layer_forward(*args, workspace=ws)
    head = ws.buf[:E.WORKSPACE_SYNC_BYTES].clone()
    assert head.any() and torch.equal(ws.get(FP8, 1, 4096, 16, 1024)[:E.WORKSPACE_SYNC_BYTES], head)


def test_sync_bytes_match_the_header():
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "epilora.h")).read()
    assert int(re.search(r"#define EPILORA_WORKSPACE_SYNC_BYTES (\d+)", text)[1]) == E.WORKSPACE_SYNC_BYTES
