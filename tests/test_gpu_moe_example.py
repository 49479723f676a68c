"""The example layer: it runs, and its parts put together are the mixture's formula in 64 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from precision_gemm_token_gb300 import moe as M

from . import moe_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def mixture(x, ids, weights, w):
    """(the experts' sum, its bound) from the inner rows that experts_up gives."""
    codes, scale = M.experts_up(x, ids, w)
    return U.down_expected(codes.cpu().numpy().reshape(-1, w.inner), scale.cpu().numpy(), ids.cpu().numpy(),
                           weights.cpu().numpy(), w.down.cpu().numpy(), w.down_scale.cpu().numpy())


@pytest.mark.parametrize("tokens", [1, 7, 300])
def test_the_layer(example, tokens):
    layer = example.MoeLayer(hidden=256, inner=208, experts=12, groups=3)
    x = U.activations(tokens, 256, seed=tokens).cuda()
    y = layer(x)
    ids, weights = layer.route(x)
    want_ids, want_w = O.route((x.float() @ layer.router.T).cpu().numpy(), 4, bias=layer.bias.cpu().numpy(),
                               scoring="sigmoid", groups=3, top_groups=2, group_best=2, scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    U.close(U.f64(weights), want_w, 2.0 ** -16 * np.abs(want_w))
    a, off_a = mixture(x, ids, weights, layer.experts)
    b, off_b = mixture(x, torch.zeros(tokens, 1, dtype=torch.int32, device="cuda"), torch.ones(tokens, 1, device="cuda"),
                       layer.shared)
    # (the two sums are bf16, and so is theirs)
    bound = off_a + off_b
    U.close(U.f64(y), a + b, bound + U.BF16 * (np.abs(a + b) + bound))
    assert int(layer.status) == 0


def test_decoding_replays(example):
    layer = example.MoeLayer(hidden=256, inner=208, experts=12, groups=3)
    dec = example.Decoder(layer, 8, 256)
    for n in (8, 3, 1):
        x = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
        x[:n] = U.activations(n, 256, seed=n).cuda()
        dec.x.zero_()
        assert torch.equal(dec.step(x[:n]), layer(x)[:n])


def test_it_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["moe_layer.py", "--tokens", "40"])
    example.main()
    assert "status 0" in capsys.readouterr().out
