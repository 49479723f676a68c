"""Choices that 64 bits cannot tell apart: scores that a sigmoid's 1 or a bias swallows go by their logits."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from precision_gemm_token_gb300 import moe as M

pytestmark = pytest.mark.gpu


def chosen(logits, top, **kw):
    ids, weights = M.route(torch.from_numpy(logits).cuda(), top, **kw)
    cpu = {k: (v.cpu().numpy() if torch.is_tensor(v) else v) for k, v in kw.items()}
    want, w = O.route(logits, top, **cpu)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert np.allclose(weights.cpu().numpy(), w, rtol=2.0 ** -16, atol=1e-37)
    return ids.cpu().numpy()


def swallowed(e, scoring, seed):
    """Distinct logits of which at least 40 have scores that no 64-bit sum with a bias of the order of 1 shows."""
    g = np.random.default_rng(seed)
    l = np.zeros((5, e), np.float32)
    for t in range(5):
        if scoring == "sigmoid":
            l[t] = g.permutation(np.linspace(41.0, 400.0, e))       # 1 - s < 2^-59
        else:
            l[t] = g.permutation(np.linspace(-400.0, -60.0, e))     # beside a 0: s < 2^-86
            l[t, g.integers(e)] = 0.0
    return l


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [0.0, 0.25, -1.0, 3.0])
@pytest.mark.parametrize("e,top", [(2, 2), (33, 5), (64, 8), (128, 32), (256, 8), (512, 10), (1000, 32)])
def test_equal_biases(e, top, bias, scoring):
    l = swallowed(e, scoring, e)
    want = np.argsort(-l, 1)[:, :top]                               # the order of the scores
    b = torch.full((e,), bias).cuda()
    for logits in (l, l[:, ::-1].copy()):
        ids = chosen(logits, top, scoring=scoring, bias=b)
        assert np.array_equal(ids, want if logits is l else np.argsort(-logits, 1)[:, :top])


def test_few_swallowed_among_others():
    """Two or three equal sums beside ordinary ones: told apart a lane each, not as a whole token."""
    g = np.random.default_rng(1)
    l = g.standard_normal((40, 96)).astype(np.float32)
    for t in range(40):
        at = g.choice(96, 3, replace=False)
        l[t, at] = np.array([40.0, 45.0, 41.0], np.float32)[g.permutation(3)]
    ids = chosen(l, 6, scoring="sigmoid", bias=torch.full((96,), 0.05).cuda())
    assert np.array_equal(ids, np.argsort(-l, 1)[:, :6])


def test_equal_logits_still_go_by_index():
    l = np.full((3, 70), 50.0, np.float32)
    l[1, 3], l[1, 66] = 60.0, 60.0
    l[2, 40:] = 45.0
    ids = chosen(l, 4, scoring="sigmoid", bias=torch.zeros(70).cuda())
    assert ids.tolist() == [[0, 1, 2, 3], [3, 66, 0, 1], [0, 1, 2, 3]]


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_groups_and_unequal_biases(scoring):
    l = swallowed(64, scoring, 5)
    g = np.random.default_rng(2)
    steps = torch.from_numpy(g.choice([0.25, 0.5], 64).astype(np.float32)).cuda()      # two kinds of equal sums
    chosen(l, 8, scoring=scoring, bias=steps)
    for best in (1, 2):
        for b in (torch.full((64,), 0.5).cuda(), steps):
            chosen(l, 8, scoring=scoring, bias=b, groups=8, top_groups=3, group_best=best)
