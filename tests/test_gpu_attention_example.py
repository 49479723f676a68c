"""The example layer: its steps (prompts, then decoding beside a chunk) against
attention in 64 bits over what the cache holds, and the attention of a whole
prompt against the same prompt through the cache."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import attention_oracle as AO
from oracle import fpformats as F
from precision_gemm_token_gb300 import attention as A

from .attention_util import assert_attention, ensure_lib, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    ensure_lib()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def held(layer, name, what):
    """A sequence's keys or values [tokens, kv_heads, dim] as float64, from the cache's pages."""
    pool = layer.cache.k if what == "k" else layer.cache.v
    scale = layer.cache.k_scale if what == "k" else layer.cache.v_scale
    t = pool[torch.tensor(layer.pages[name]).cuda()].transpose(1, 2).reshape(-1, layer.kv_heads, layer.dim)
    t = t[:layer.length[name]]
    if scale is None:
        return f64(t)
    return F.e4m3_decode(t.cpu().numpy()).astype(np.float64) * f64(scale)[None, :, None]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_example_steps(example, kv):
    layer = example.AttentionLayer(hidden=512, heads=8, kv_heads=2, dim=64 if kv == "bf16" else 128, pages=64, kv=kv)
    g = torch.Generator(device="cuda").manual_seed(3)
    steps = [[("a", 70), ("b", 5), ("c", 1)], [("a", 1), ("d", 130), ("c", 2)], [("a", 1), ("b", 1), ("c", 1), ("d", 1)]]
    for seqs in steps:
        tokens = sum(n for _, n in seqs)
        x = torch.randn(tokens, layer.hidden, generator=g, device="cuda").to(torch.bfloat16)
        tenant = (torch.arange(tokens, dtype=torch.int32) % 5 - 1).cuda()
        y, q, o = layer.step(x, tenant, layer.plan(seqs))
        assert int(layer.status.item()) == 0
        assert y.shape == x.shape and bool(torch.isfinite(y).all()) and float(y.float().abs().mean()) > 0
        at = 0
        for name, n in seqs:
            k, v = held(layer, name, "k"), held(layer, name, "v")
            positions = np.arange(layer.length[name] - n, layer.length[name])
            w, lse, bounds = AO.attention_rows(f64(q[at:at + n]), k, v, positions, layer.dim ** -0.5)
            assert_attention(o[at:at + n], None, w, lse, *bounds, what=(name, seqs), fmt=kv)
            at += n


def test_example_prompt_agrees_with_cache(example):
    """A bf16 cache holds the keys and values as they are: both calls are the
    same attention, each within its bound of the 64-bit one."""
    layer = example.AttentionLayer(hidden=512, heads=8, kv_heads=2, dim=128, pages=64)
    n = 201
    x = torch.randn(n, layer.hidden, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    plan = layer.plan([("a", n)])
    _, q, o = layer.step(x.to(torch.bfloat16), torch.zeros(n, dtype=torch.int32, device="cuda"), plan)
    k, v = (torch.from_numpy(held(layer, "a", c)).cuda().to(torch.bfloat16) for c in "kv")
    whole = A.prompt_attention(q, k, v, plan[0], workspace=layer.attn_ws, status=layer.status)
    assert int(layer.status.item()) == 0
    w, lse, bounds = AO.attention_rows(f64(q), f64(k), f64(v), np.arange(n), layer.dim ** -0.5)
    assert_attention(o, None, w, lse, *bounds, what="cache")
    assert_attention(whole, None, w, lse, *bounds, what="prompt")


def test_example_main(example, capsys, monkeypatch):
    for kv in ("bf16", "e4m3"):
        monkeypatch.setattr("sys.argv", ["attention_layer.py", "--kv", kv, "--decode", "3"])
        example.main()
    assert "lengths {'a': 505, 'c': 216, 'd': 304}" in capsys.readouterr().out
