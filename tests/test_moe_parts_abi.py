"""Host-side checks of the experts' calls that keep the outputs of the experts in fp32: workspace sizes and refusals,
before anything is enqueued (fake addresses, only where no device exists to launch on)."""
import pytest
import torch

import precision_gemm_token_gb300 as E
from precision_gemm_token_gb300 import moe as M

FAKE = 0x10000
INVALID, UNSUP, WS = E.EPILORA_ERR_INVALID_ARG, E.EPILORA_ERR_UNSUPPORTED, E.EPILORA_ERR_WORKSPACE
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only where nothing can launch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    E.build()
    return E.load()


def test_workspace_bytes():
    size = (4, 2, 8, 256, 128)
    more = 8 * 256 * 2                                  # fp32 instead of bf16: two bytes more per slot and column
    for what in (E.MOE_DOWN, E.MOE_UP | E.MOE_DOWN):
        assert E.epilora_moe_workspace_bytes(what | E.MOE_F32_PARTS, *size) == \
            E.epilora_moe_workspace_bytes(what, *size) + more
    assert E.epilora_moe_workspace_bytes(E.MOE_UP | E.MOE_F32_PARTS, *size) == 0
    assert E.epilora_moe_workspace_bytes(E.MOE_F32_PARTS, *size) == 0
    assert E.epilora_moe_workspace_bytes(8 | E.MOE_DOWN, *size) == 0


def call(which, **kw):
    a = dict(T=4, k=2, E=8, H=256, I=128, X=FAKE, ldx=256, ids=FAKE, w=FAKE, up=FAKE, ups=FAKE, down=FAKE, downs=FAKE,
             hq=FAKE, hs=FAKE, Y=FAKE, ldy=256, ws=FAKE, n=1 << 30, st=None)
    a.update(kw)
    size, end = (a["T"], a["k"], a["E"], a["H"], a["I"]), (a["ws"], a["n"], a["st"], 0)
    if which == "down":
        return E.epilora_moe_experts_down_f32(*size, a["hq"], a["hs"], a["ids"], a["w"], a["down"], a["downs"], a["Y"],
                                              a["ldy"], *end)
    return E.epilora_moe_experts_f32(*size, a["X"], a["ldx"], a["ids"], a["w"], a["up"], a["ups"], a["down"], a["downs"],
                                     a["Y"], a["ldy"], *end)


@no_gpu
@pytest.mark.parametrize("which", ["down", "both"])
def test_refusals(which):
    for kw, want in ((dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(I=8), INVALID), (dict(E=1025), UNSUP),
                     (dict(ids=None), INVALID), (dict(w=FAKE + 2), INVALID), (dict(down=FAKE + 8), INVALID),
                     (dict(Y=None), INVALID), (dict(ldy=260), INVALID), (dict(st=FAKE + 2), INVALID),
                     (dict(ws=None), WS), (dict(ws=FAKE + 64), WS), (dict(T=0, Y=None, ids=None, ws=None), E.EPILORA_OK)):
        assert call(which, **kw) == want, kw
    what = (E.MOE_DOWN if which == "down" else E.MOE_UP | E.MOE_DOWN)
    # room for bf16 parts is not enough
    assert call(which, n=E.epilora_moe_workspace_bytes(what, 4, 2, 8, 256, 128)) == WS


def test_helpers_refuse_other_types():
    for dtype in (torch.float16, torch.float64, None, "fp32"):
        with pytest.raises(E.EpiloraError):
            M._parts(dtype)
