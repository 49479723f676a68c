"""The attention workspace's life: made before or under a graph capture, used
on several streams, shared between head sizes. Cut sequences, whose pieces
meet in the workspace, in every call."""
import pytest
import torch

import precision_gemm_token_gb300 as E
from precision_gemm_token_gb300 import attention as A

from .attention_util import Batch, ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.fixture
def dirty():
    """A graph memory pool, and cached memory, whose free blocks hold ones:
    what a call takes from them without filling it is not zero by chance."""
    pool = torch.cuda.graph_pool_handle()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, pool=pool):
        x = [torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        del x
    g.replay()
    x = [torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del x
    yield pool
    del g


class Call:
    """One attention call whose sequence is cut between blocks."""

    def __init__(self, n, dim=128, seed=0):
        self.b = Batch([(n, 9000)], 8, 2, dim, seed=seed)
        self.args = self.b.dev("q", "q_start", "kv_len", "table")
        self.ref = self.run(A.AttentionWorkspace("cuda")).clone()
        torch.cuda.synchronize()

    def run(self, ws, stream=None, out=None):
        q, start, length, table = self.args
        if out is None:
            out = torch.full_like(q, 7.0)
            torch.cuda.synchronize()
        return A.paged_attention(q, self.b.cache, start, length, table, max_new=q.shape[0], out=out, workspace=ws,
                                 stream=stream)


def captured(call, ws, pool):
    """(graph, its output, workspace); ws: a workspace, or a function that makes one under the capture."""
    out = torch.full_like(call.ref, 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, pool=pool):
        w = ws() if callable(ws) else ws
        call.run(w, out=out)
    return g, out, w


def replayed(g, out):
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("n", [1, 40])
def test_first_used_under_capture(n, dirty):
    """An eager call before the first replay, and the replays, are right."""
    call = Call(n)
    ws = A.AttentionWorkspace("cuda")
    g, out, _ = captured(call, ws, dirty)
    assert torch.equal(call.run(ws), call.ref)
    assert torch.equal(replayed(g, out), call.ref)
    assert torch.equal(call.run(ws), call.ref)
    assert torch.equal(replayed(g, out), call.ref)


@pytest.mark.parametrize("n", [1, 40])
def test_two_graphs_before_a_replay(n, dirty):
    """The second captured graph is replayed first."""
    call = Call(n)
    ws = A.AttentionWorkspace("cuda")
    (g1, out1, _), (g2, out2, _) = captured(call, ws, dirty), captured(call, ws, dirty)
    assert torch.equal(replayed(g2, out2), call.ref)
    assert torch.equal(replayed(g1, out1), call.ref)
    assert torch.equal(replayed(g2, out2), call.ref)


@pytest.mark.parametrize("n", [1, 40])
def test_made_under_capture(n, dirty):
    """A workspace made inside a capture serves that graph, and, once made,
    eager calls and other graphs before its replay."""
    call = Call(n)
    g, out, ws = captured(call, lambda: A.AttentionWorkspace("cuda"), dirty)
    assert torch.equal(call.run(ws), call.ref)
    g2, out2, _ = captured(call, ws, dirty)
    for _ in range(2):
        assert torch.equal(replayed(g2, out2), call.ref)
        assert torch.equal(replayed(g, out), call.ref)
        assert torch.equal(call.run(ws), call.ref)


@pytest.mark.parametrize("n", [1, 40])
def test_no_workspace_under_capture(n, dirty):
    call = Call(n)
    g, out, _ = captured(call, lambda: None, dirty)
    for _ in range(2):
        assert torch.equal(replayed(g, out), call.ref)
    assert torch.equal(call.run(None), call.ref)


def test_first_used_on_another_stream(dirty):
    """Zero before the first call, whichever stream that goes to."""
    call = Call(1)
    for _ in range(5):
        s = torch.cuda.Stream()
        busy = torch.randn(2048, 2048, device="cuda")
        out = torch.full_like(call.ref, 7.0)
        torch.cuda.synchronize()
        for _ in range(20):
            busy = busy @ busy * 1e-3      # the current stream is behind when the workspace is made
        ws = A.AttentionWorkspace("cuda")
        call.run(ws, stream=s, out=out)
        s.synchronize()
        assert torch.equal(out, call.ref)
        torch.cuda.synchronize()


def test_head_sizes_share_a_workspace():
    calls = [Call(1, 128), Call(40, 64, seed=1), Call(1, 64, seed=2), Call(40, 128, seed=3)]
    ws = A.AttentionWorkspace("cuda")
    for _ in range(3):
        for c in calls:
            assert torch.equal(c.run(ws), c.ref)


def test_workspace_device():
    """The device is settled when the workspace is made; one that is no CUDA
    device is refused."""
    ws = A.AttentionWorkspace("cuda")
    assert ws.device == torch.device("cuda", torch.cuda.current_device())
    for device in ("cpu", torch.device("meta")):
        with pytest.raises(E.EpiloraError, match="workspace"):
            A.AttentionWorkspace(device)
