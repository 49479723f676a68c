"""Which device an attention workspace belongs to. No GPU: the current device
and the tensors' devices are stand-ins."""
import pytest
import torch

import precision_gemm_token_gb300 as E
from precision_gemm_token_gb300 import attention as A


@pytest.fixture(autouse=True)
def no_allocation(monkeypatch):
    monkeypatch.setattr(A.AttentionWorkspace, "_make", lambda self: None)


class OnDevice:
    """A tensor as far as the workspace looks at one."""

    device = torch.device("cpu")

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


def test_device_without_an_index_is_the_current_one(monkeypatch):
    for current in (0, 1):
        monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
        assert A.AttentionWorkspace("cuda").device == torch.device("cuda", current)
        assert A.AttentionWorkspace("cuda:0").device == torch.device("cuda", 0)


def test_workspace_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for made in ("cuda", "cuda:0"):
        with pytest.raises(E.EpiloraError, match="workspace: on cuda:0"):
            A._workspace(A.AttentionWorkspace(made), OnDevice(1), 128, 0, None)


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_other_devices_are_refused(device):
    with pytest.raises(E.EpiloraError, match="workspace: a CUDA device"):
        A.AttentionWorkspace(device)


def test_bytes_to_zero():
    """The counters: whole 256-byte units, a small part of the workspace."""
    E.build()
    n = E.epilora_attention_workspace_zero_bytes()
    assert 0 < n <= 1 << 16 and n % 256 == 0
    assert E.epilora_attention_workspace_bytes(128) > E.epilora_attention_workspace_bytes(64) > n


@pytest.mark.parametrize("dim", [64, 128])
def test_a_call_without_a_workspace_fills_the_counters_alone(dim, monkeypatch):
    E.build()
    made, empty = [], torch.empty

    def ones(*a, **kw):
        made.append(empty(*a, **kw).fill_(255))
        return made[-1]

    monkeypatch.setattr(torch, "empty", ones)
    buf, address, size = A._workspace(None, OnDevice(0), dim, 0, None)
    n = E.epilora_attention_workspace_zero_bytes()
    assert buf is made[0] and address == buf.data_ptr() and size == E.epilora_attention_workspace_bytes(dim)
    assert not buf[:n].any() and (buf[n:] == 255).all()
