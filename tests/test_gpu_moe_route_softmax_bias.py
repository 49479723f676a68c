"""Softmax scores with a bias: many tokens, and choices that lie closer than the scores' 32-bit errors."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from precision_gemm_token_gb300 import moe as M

pytestmark = pytest.mark.gpu


def check(logits, top, bias, **kw):
    ids, weights = M.route(torch.from_numpy(logits).cuda(), top, bias=torch.from_numpy(bias).cuda(), **kw)
    want, w = O.route(logits, top, bias=bias, **kw)
    assert np.array_equal(ids.cpu().numpy(), want), np.argwhere(ids.cpu().numpy() != want)[:4]
    # logits of up to 12 in size: an exponential's argument is off by 24 u of it, sums and quotients by less than 60 u
    assert (np.abs(weights.cpu().numpy() - w) <= 96 * 2.0 ** -24 * w).all()


@pytest.mark.parametrize("size", [0.05, 0.001])
@pytest.mark.parametrize("e,top", [(60, 4), (256, 8), (320, 16), (512, 16)])
def test_many_tokens(e, top, size):
    g = np.random.default_rng(e)
    logits = (1.5 * g.standard_normal((1500, e)) + 0.5 * g.standard_normal(e)).astype(np.float32)
    check(logits, top, (size * g.standard_normal(e)).astype(np.float32))


@pytest.mark.parametrize("spread", [0.0, 2.0 ** -31, 2.0 ** -27, 2.0 ** -23])
@pytest.mark.parametrize("e,top", [(40, 5), (128, 8), (256, 8), (512, 16), (1024, 32)])
def test_choices_closer_than_the_scores_errors(e, top, spread):
    """Each bias is what its score lacks to one small sum, and up to `spread` more: sums as small as the scores, whose order
    the scores' roundings turn round where 32 bits are believed."""
    g = np.random.default_rng(e + top)
    z = (0.7 * g.standard_normal(e)).astype(np.float32)
    s = np.exp(z.astype(np.float64) - z.max())
    s /= s.sum()
    bias = (1.5 * s.max() - s + spread * g.random(e)).astype(np.float32)
    logits = np.tile(z, (6, 1))
    logits[3:] = z + np.float32(2.0 ** -18) * g.standard_normal((3, e)).astype(np.float32)
    check(logits, top, bias)
    if e % 8 == 0 and top <= e // 8 * 3:
        check(logits, top, bias, groups=8, top_groups=3, group_best=2)
