"""Host-side argument checks of the operators in 8-bit blocks and of the
mixture of experts: every call below is refused before anything is enqueued
(fake, never dereferenced addresses; only where no device exists to launch on),
and the oracle's own pins."""
import numpy as np
import pytest
import torch

import precision_gemm_token_gb300 as E
from oracle import fpformats as F
from oracle import moe_oracle as O
from precision_gemm_token_gb300 import blocks as B
from precision_gemm_token_gb300 import moe as M

FAKE = 0x10000
INVALID, UNSUP, WS = E.EPILORA_ERR_INVALID_ARG, E.EPILORA_ERR_UNSUPPORTED, E.EPILORA_ERR_WORKSPACE
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only where nothing can launch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    E.build()
    return E.load()


def quant(fn="epilora_block_quant", **kw):
    a = dict(X=FAKE, M=4, K=256, ldx=256, Xq=FAKE, s=FAKE, ld=4)
    a.update(kw)
    if fn == "epilora_block_quant":
        return E.epilora_block_quant(a["X"], a["M"], a["K"], a["ldx"], a["Xq"], a["s"], a["ld"], 0)
    return E.epilora_block_quant_weight(a["X"], a["M"], a["K"], a["ldx"], a["Xq"], a["s"], 0)


BAD_QUANT = [dict(M=-1), dict(K=0), dict(K=8), dict(K=250, ldx=256), dict(ldx=248), dict(ldx=260), dict(X=None),
             dict(X=FAKE + 8), dict(Xq=None), dict(Xq=FAKE + 4), dict(s=None), dict(s=FAKE + 2)]


@no_gpu
@pytest.mark.parametrize("kw", BAD_QUANT)
def test_quantizers(kw):
    assert quant(**kw) == INVALID and quant("epilora_block_quant_weight", **kw) == INVALID


@no_gpu
def test_quantizer_scale_stride_and_nothing_to_do():
    assert quant(ld=3) == INVALID
    assert quant(M=0, X=None, Xq=None, s=None, ld=0) == E.EPILORA_OK
    assert quant("epilora_block_quant_weight", M=0, X=None, Xq=None, s=None) == E.EPILORA_OK


def matmul(**kw):
    a = dict(M=4, N=100, K=256, Xq=FAKE, xs=FAKE, ld=4, Wq=FAKE, ws=FAKE, Y=FAKE, ldy=100, st=None)
    a.update(kw)
    return E.epilora_block_matmul(a["M"], a["N"], a["K"], a["Xq"], a["xs"], a["ld"], a["Wq"], a["ws"], a["Y"], a["ldy"],
                                  a["st"], 0)


def linear(**kw):
    a = dict(M=4, N=100, K=256, X=FAKE, ldx=256, Wq=FAKE, ws=FAKE, Y=FAKE, ldy=100, w=FAKE, n=1 << 20, st=None)
    a.update(kw)
    return E.epilora_block_linear(a["M"], a["N"], a["K"], a["X"], a["ldx"], a["Wq"], a["ws"], a["Y"], a["ldy"], a["w"],
                                  a["n"], a["st"], 0)


BAD_PRODUCT = [dict(M=-1), dict(N=0), dict(K=24, ldx=32), dict(Wq=None), dict(Wq=FAKE + 8), dict(ws=None), dict(ws=FAKE + 1),
               dict(Y=None), dict(Y=FAKE + 1), dict(ldy=99), dict(st=FAKE + 2)]


@no_gpu
@pytest.mark.parametrize("kw", BAD_PRODUCT)
def test_products(kw):
    assert linear(**kw) == INVALID
    kw.pop("ldx", None)
    assert matmul(**kw) == INVALID


@no_gpu
def test_products_own_arguments():
    for kw in (dict(Xq=None), dict(Xq=FAKE + 8), dict(xs=None), dict(xs=FAKE + 2), dict(ld=3)):
        assert matmul(**kw) == INVALID
    for kw in (dict(X=None), dict(X=FAKE + 8), dict(ldx=250), dict(ldx=260)):
        assert linear(**kw) == INVALID
    need = E.epilora_block_linear_workspace_bytes(4, 256)
    assert need == 1024 + 256
    for kw in (dict(w=None), dict(w=FAKE + 128), dict(n=need - 1)):
        assert linear(**kw) == WS
    assert E.epilora_block_linear_workspace_bytes(-1, 256) == 0 and E.epilora_block_linear_workspace_bytes(4, 24) == 0
    assert matmul(M=0, Xq=None, xs=None, ld=0, Wq=None) == E.EPILORA_OK and linear(M=0, X=None, w=None, n=0) == E.EPILORA_OK


def route(**kw):
    a = dict(T=4, E=64, k=8, l=FAKE, fmt=0, ld=64, bias=None, score=0, g=1, tg=1, gb=1, scale=1.0, ids=FAKE, w=FAKE)
    a.update(kw)
    return E.epilora_moe_route(a["T"], a["E"], a["k"], a["l"], a["fmt"], a["ld"], a["bias"], a["score"], a["g"], a["tg"],
                               a["gb"], True, a["scale"], a["ids"], a["w"], 0)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(ld=63), INVALID), (dict(fmt=2), INVALID),
    (dict(score=2), INVALID), (dict(g=0), INVALID), (dict(g=5), INVALID), (dict(tg=0), INVALID), (dict(tg=2), INVALID),
    (dict(gb=0), INVALID), (dict(gb=3), INVALID), (dict(k=65), INVALID), (dict(g=8, tg=1, k=9), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(l=None), INVALID),
    (dict(l=FAKE + 2), INVALID), (dict(l=FAKE + 1, fmt=1), INVALID), (dict(bias=FAKE + 2), INVALID), (dict(ids=None), INVALID),
    (dict(w=FAKE + 2), INVALID), (dict(E=2048, ld=2048), UNSUP), (dict(k=33), UNSUP), (dict(g=64, tg=64), UNSUP)])
def test_route(kw, want):
    assert route(**kw) == want


@no_gpu
def test_route_nothing_to_do():
    assert route(T=0, l=None, ids=None, w=None) == E.EPILORA_OK


def experts(which, **kw):
    a = dict(T=4, k=2, E=8, H=256, I=128, X=FAKE, ldx=256, ids=FAKE, w=FAKE, up=FAKE, ups=FAKE, down=FAKE, downs=FAKE, hq=FAKE,
             hs=FAKE, Y=FAKE, ldy=256, ws=FAKE, n=1 << 30, st=None)
    a.update(kw)
    size = (a["T"], a["k"], a["E"], a["H"], a["I"])
    end = (a["ws"], a["n"], a["st"], 0)
    if which == "up":
        return E.epilora_moe_experts_up(*size, a["X"], a["ldx"], a["ids"], a["up"], a["ups"], a["hq"], a["hs"], *end)
    if which == "down":
        return E.epilora_moe_experts_down(*size, a["hq"], a["hs"], a["ids"], a["w"], a["down"], a["downs"], a["Y"], a["ldy"],
                                          *end)
    return E.epilora_moe_experts(*size, a["X"], a["ldx"], a["ids"], a["w"], a["up"], a["ups"], a["down"], a["downs"], a["Y"],
                                 a["ldy"], *end)


@no_gpu
@pytest.mark.parametrize("which", ["up", "down", "both"])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(E=0), INVALID), (dict(H=24, ldx=32), INVALID), (dict(I=8), INVALID),
    (dict(I=0), INVALID), (dict(E=1025), UNSUP), (dict(T=1 << 29, k=2), UNSUP), (dict(ids=None), INVALID),
    (dict(ids=FAKE + 2), INVALID), (dict(st=FAKE + 2), INVALID), (dict(ws=None), WS), (dict(ws=FAKE + 64), WS), (dict(n=100), WS)])
def test_experts(which, kw, want):
    assert experts(which, **kw) == want


@no_gpu
def test_experts_own_arguments():
    own = {"up": ["X", "up", "ups", "hq", "hs"], "down": ["hq", "hs", "w", "down", "downs", "Y"],
           "both": ["X", "w", "up", "ups", "down", "downs", "Y"]}
    for which, names in own.items():
        for name in names:
            assert experts(which, **{name: None}) == INVALID, (which, name)
            assert experts(which, **{name: FAKE + 2}) == INVALID, (which, name)
    for which in ("up", "both"):
        assert experts(which, ldx=255) == INVALID and experts(which, ldx=260) == INVALID
    for which in ("down", "both"):
        assert experts(which, ldy=255) == INVALID and experts(which, ldy=260) == INVALID
    for which in own:
        assert experts(which, T=0, X=None, ids=None, ws=None, Y=None, hq=None) == E.EPILORA_OK


def test_workspace_bytes():
    r = lambda n: -(-n // 256) * 256  # noqa: E731
    plan = r(9 * 4) + 2 * r(8 * 4)
    up, down = r(8 * 256) + r(2 * 8 * 4), r(8 * 128) + r(8 * 4) + r(8 * 256 * 2)
    size = (4, 2, 8, 256, 128)
    assert E.epilora_moe_workspace_bytes(E.MOE_UP, *size) == plan + up
    assert E.epilora_moe_workspace_bytes(E.MOE_DOWN, *size) == plan + down
    assert E.epilora_moe_workspace_bytes(E.MOE_UP | E.MOE_DOWN, *size) == plan + up + down
    for what, bad in ((0, size), (4, size), (1, (4, 2, 2000, 256, 128)), (1, (4, 0, 8, 256, 128)), (1, (4, 2, 8, 250, 128))):
        assert E.epilora_moe_workspace_bytes(what, *bad) == 0


def test_helpers_refuse_what_is_not_on_a_device():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(E.EpiloraError):
        B.block_quant(x)
    with pytest.raises(E.EpiloraError):
        M.route(torch.zeros(4, 8), 2)
    with pytest.raises(E.EpiloraError):
        B.BlockWorkspace("cpu")
    with pytest.raises(E.EpiloraError):
        B.BlockWeight(torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(2, 1))
    with pytest.raises(E.EpiloraError):
        B.BlockWeight(torch.zeros(4, 8), torch.zeros(1, 1))
    codes, s = torch.zeros(2, 2, 16, 32, dtype=torch.uint8), torch.zeros(2, 2, 1, 1)
    down, ds = torch.zeros(2, 32, 16, dtype=torch.uint8), torch.zeros(2, 1, 1)
    M.ExpertWeights(codes, s, down, ds)
    for bad in ((codes[:, :1], s[:, :1], down, ds), (codes, s[:1], down, ds), (codes, s, down.transpose(1, 2), ds),
                (codes, s, down, ds.double()), (codes.int(), s, down, ds)):
        with pytest.raises(E.EpiloraError):
            M.ExpertWeights(*bad)


def test_oracle_quantizer():
    x = np.zeros((2, 300), np.float32)
    x[0, 0], x[0, 1], x[0, 128:256] = 448.0, 1.0, 2.0
    codes, scale = O.quant_rows(x)
    assert scale.shape == (3, 2) and scale[0, 0] == 1.0 and scale[1, 0] == np.float32(2) / np.float32(448)
    v = F.e4m3_decode(codes)
    assert v[0, 0] == 448 and v[0, 1] == 1 and (v[0, 128:256] == 448).all() and (v[0, 256:] == 0).all() and (v[1] == 0).all()
    assert (scale[:, 1] == np.float32(1e-12) / np.float32(448)).all()
    g = np.random.default_rng(0)
    w = g.standard_normal((200, 300)).astype(np.float32)
    c, s = O.quant_weight(w)
    assert s.shape == (2, 3)
    assert np.abs(O.values_weight(c, s) - w).max() <= 2.0 ** -4 * np.abs(w).max()
    for i in range(2):
        for b in range(3):
            part = np.s_[i * 128:(i + 1) * 128, b * 128:(b + 1) * 128]
            assert np.abs(F.e4m3_decode(c[part])).max() == 448 and s[i, b] == np.abs(w[part]).max() / np.float32(448)


def test_oracle_route():
    z = np.log(np.array([[1.0, 2.0, 4.0, 8.0]]))
    ids, w = O.route(z, 2)
    assert ids.tolist() == [[3, 2]] and np.allclose(w, [[8 / 12, 4 / 12]])
    ids, w = O.route(z, 2, renormalize=False, scale=3.0)
    assert np.allclose(w, [[8 / 15 * 3, 4 / 15 * 3]])
    ids, w = O.route(z, 1, bias=np.array([1.0, 0, 0, 0]))
    assert ids.tolist() == [[0]] and np.allclose(w, [[1.0]])
    ids, _ = O.route(z, 2, groups=2, top_groups=1)
    assert ids.tolist() == [[3, 2]]
    # by the two best the first pair wins, by the best alone the second
    z = np.array([[1.0, 1.0, 1.5, -9.0]])
    assert O.route(z, 1, groups=2, group_best=2, scoring="sigmoid")[0].tolist() == [[0]]
    assert O.route(z, 1, groups=2, group_best=1, scoring="sigmoid")[0].tolist() == [[2]]
    ids, w = O.route(np.array([[-np.inf, np.nan, 0.0], [-np.inf] * 3]), 2)
    assert ids.tolist() == [[2, -1], [-1, -1]] and w.tolist() == [[1.0, 0.0], [0.0, 0.0]]
    assert O.route(np.zeros((1, 5)), 3)[0].tolist() == [[0, 1, 2]]
