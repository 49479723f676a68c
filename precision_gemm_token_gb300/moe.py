"""Tensor-level helpers over the C ABI's mixture-of-experts calls: routing,
and the experts' gated MLPs in 8-bit blocks (see `blocks`). No arithmetic of
the operators happens here.

    w = quantize_experts(gate, up, down)               # once; or ExpertWeights of a checkpoint's codes and scales
    ids, weights = route(logits, 8, bias=bias, scoring="sigmoid", groups=8, top_groups=4, group_best=2)
    y = experts(x, ids, weights, w, workspace=ws)      # ws: blocks.BlockWorkspace
    h, hs = experts_up(x, ids, w)                      # the two halves of it
    y = experts_down(h, hs, ids, weights, w)
"""
from __future__ import annotations

from functools import lru_cache
from typing import Optional

import torch

from . import _binding as E
from .blocks import (_BF16, _F32, _I32, _U8, BlockWorkspace, _array, _bad, _blocks, _lib, _made, _matrix, _out, _room,
                     _new, _quantize_weight, _start, _status)

_SCORING = {"softmax": E.SCORE_SOFTMAX, "sigmoid": E.SCORE_SIGMOID}
_bytes = lru_cache(1024)(E.epilora_moe_workspace_bytes)       # asked of the library once per shape
_LOGITS = {torch.float32: E.LOGITS_F32, torch.bfloat16: E.LOGITS_BF16}


def route(logits, top: int, bias=None, scoring: str = "softmax", groups: int = 1, top_groups: int = 1,
          group_best: int = 1, renormalize: bool = True, scale: float = 1.0, ids=None, weights=None, stream=None):
    """The `top` experts of each token and their weights from the router's
    logits [tokens, experts] (fp32 or bf16, rows that do not overlap): (ids
    int32 [tokens, top], weights fp32 [tokens, top]). `bias` (fp32 [experts]) is
    added to the scores for the choice alone; with groups > 1 the experts come
    from the `top_groups` groups whose `group_best` largest choices sum to the
    most. epilora_moe_route has the details."""
    dev, raw, given = _start(logits, stream)
    fmt, how = _LOGITS.get(logits.dtype), _SCORING.get(scoring)
    if fmt is None or how is None:
        _bad("route: fp32 or bf16 logits, scoring 'softmax' or 'sigmoid' wanted")
    at, T, n, _ = _matrix(logits, logits.dtype, dev, "logits")
    ld = logits.stride(0) if T > 1 else n
    b_at = None if bias is None else _array(bias, _F32, (n,), dev, "bias")
    shape = (T, top if top > 0 else 0)
    ids, i_at = _made(ids, logits, shape, _I32, dev, given, "ids")
    weights, w_at = _made(weights, logits, shape, _F32, dev, given, "weights")
    rc = _lib().epilora_moe_route(T, n, top, at, fmt, ld, b_at, how, groups, top_groups, group_best,
                                  1 if renormalize else 0, scale, i_at, w_at, raw)
    if rc:
        E.check(rc, "route")
    return ids, weights


class ExpertWeights:
    """The experts' gated MLPs: E4M3 codes gate_up uint8 [experts, 2, inner,
    hidden] (gate, then up) and down [experts, hidden, inner], with fp32 scales
    of their 128 x 128 blocks [experts, 2, ceil(inner / 128), ceil(hidden /
    128)] and [experts, ceil(hidden / 128), ceil(inner / 128)]. The tensors
    stay the caller's."""

    def __init__(self, gate_up, gate_up_scale, down, down_scale):
        if gate_up.dim() != 4 or gate_up.shape[1] != 2:
            _bad("gate_up: uint8 [experts, 2, inner, hidden] wanted")
        n, _, inner, hidden = gate_up.shape
        dev = gate_up.get_device()
        self.up_at = _array(gate_up, _U8, (n, 2, inner, hidden), dev, "gate_up")
        self.up_scale_at = _array(gate_up_scale, _F32, (n, 2, _blocks(inner), _blocks(hidden)), dev, "gate_up_scale")
        self.down_at = _array(down, _U8, (n, hidden, inner), dev, "down")
        self.down_scale_at = _array(down_scale, _F32, (n, _blocks(hidden), _blocks(inner)), dev, "down_scale")
        self.gate_up, self.gate_up_scale, self.down, self.down_scale = gate_up, gate_up_scale, down, down_scale
        self.experts, self.inner, self.hidden, self.dev = n, inner, hidden, dev


def quantize_experts(gate, up, down, stream=None) -> ExpertWeights:
    """Load-time quantization of bf16 weights: gate and up [experts, inner,
    hidden], down [experts, hidden, inner]. Beside them it takes the memory of
    the codes and scales that it returns, no more."""
    dev, raw, given = _start(gate, stream)
    if gate.dim() != 3 or not len(gate) or up.shape != gate.shape or down.shape != (len(gate), *gate.shape[:0:-1]):
        _bad("quantize_experts: gate and up [experts, inner, hidden], down [experts, hidden, inner] wanted")
    n, inner, hidden = gate.shape
    bi, bh = _blocks(inner), _blocks(hidden)
    parts = [(_matrix(m[e], _BF16, dev, what), e, which)
             for e in range(n) for which, (m, what) in enumerate(((gate, "gate"), (up, "up"), (down, "down")))]
    gu, gus = _new(gate, (n, 2, inner, hidden), _U8, given), _new(gate, (n, 2, bi, bh), _F32, given)
    d, ds = _new(gate, (n, hidden, inner), _U8, given), _new(gate, (n, bh, bi), _F32, given)
    for at, e, which in parts:
        codes, scale = (gu[e, which], gus[e, which]) if which < 2 else (d[e], ds[e])
        _quantize_weight(*at, codes, scale, raw)
    return ExpertWeights(gu, gus, d, ds)


# what the experts' outputs are kept in until their weighted sum: (bit of the workspace's size, calls of the library)
_PARTS = {_BF16: (0, "epilora_moe_experts_down", "epilora_moe_experts"),
          _F32: (E.MOE_F32_PARTS, "epilora_moe_experts_down_f32", "epilora_moe_experts_f32")}


def _parts(dtype):
    if dtype not in _PARTS:
        _bad("parts: torch.bfloat16 or torch.float32 wanted")
    return _PARTS[dtype]


def _choices(ids, tokens, dev):
    if ids.dim() != 2 or ids.shape[0] != tokens:
        _bad(f"ids: int32 [{tokens}, top] wanted")
    return _array(ids, _I32, tuple(ids.shape), dev, "ids"), ids.shape[1]


def experts_up(x, ids, w: ExpertWeights, codes=None, scale=None, workspace: Optional[BlockWorkspace] = None,
               status=None, stream=None):
    """silu(x gate^T) * (x up^T) of each token's experts, block-quantized:
    (codes uint8 [tokens, top, inner], scale fp32 [ceil(inner / 128), tokens *
    top]). x bf16 [tokens, hidden]; ids int32 [tokens, top], negative: no
    expert, whose rows are zero."""
    dev, raw, given = _start(x, stream)
    if w.dev != dev:
        _bad("experts_up: x and the weights on different devices")
    at, T, H, ld = _matrix(x, _BF16, dev, "x", None, w.hidden)
    i_at, top = _choices(ids, T, dev)
    shape, s_shape = (T, top, w.inner), (_blocks(w.inner), T * top)
    codes, c_at = _made(codes, x, shape, _U8, dev, given, "codes")
    scale, s_at = _made(scale, x, s_shape, _F32, dev, given, "scale")
    need = _bytes(E.MOE_UP, T, top, w.experts, H, w.inner)
    buf, w_at = _room(workspace, x, need, dev, raw, given)
    rc = _lib().epilora_moe_experts_up(T, top, w.experts, H, w.inner, at, ld, i_at, w.up_at, w.up_scale_at, c_at, s_at,
                                       w_at, need, _status(status, dev), raw)
    if rc:
        E.check(rc, "experts_up")
    return codes, scale


def experts_down(codes, scale, ids, weights, w: ExpertWeights, out=None, workspace: Optional[BlockWorkspace] = None,
                 status=None, stream=None, parts=torch.bfloat16):
    """The weighted sum over a token's experts of their down projections of
    experts_up's rows: bf16 [tokens, hidden]. With `parts` bf16 each expert's
    output is rounded to it before the sum; with fp32 the sum alone is, for
    twice the traffic of the outputs (which counts in prefill batches)."""
    dev, raw, given = _start(codes, stream)
    bit, call, _ = _parts(parts)
    if w.dev != dev or codes.dim() != 3:
        _bad("experts_down: codes [tokens, top, inner] on the weights' device wanted")
    T, top = codes.shape[:2]
    c_at = _array(codes, _U8, (T, top, w.inner), dev, "codes")
    s_at = _array(scale, _F32, (_blocks(w.inner), T * top), dev, "scale")
    i_at, f_at = _array(ids, _I32, (T, top), dev, "ids"), _array(weights, _F32, (T, top), dev, "weights")
    out, o_at, ld = _out(out, codes, T, w.hidden, dev, given)
    need = _bytes(E.MOE_DOWN | bit, T, top, w.experts, w.hidden, w.inner)
    buf, w_at = _room(workspace, codes, need, dev, raw, given)
    rc = getattr(_lib(), call)(T, top, w.experts, w.hidden, w.inner, c_at, s_at, i_at, f_at, w.down_at, w.down_scale_at,
                               o_at, ld, w_at, need, _status(status, dev), raw)
    if rc:
        E.check(rc, "experts_down")
    return out


def experts(x, ids, weights, w: ExpertWeights, out=None, workspace: Optional[BlockWorkspace] = None, status=None,
            stream=None, parts=torch.bfloat16):
    """experts_up, then experts_down: y[t] = sum_j weights[t, j] *
    MLP_{ids[t, j]}(x[t]), bf16 [tokens, hidden]."""
    dev, raw, given = _start(x, stream)
    bit, _, call = _parts(parts)
    if w.dev != dev:
        _bad("experts: x and the weights on different devices")
    at, T, H, ld = _matrix(x, _BF16, dev, "x", None, w.hidden)
    i_at, top = _choices(ids, T, dev)
    f_at = _array(weights, _F32, (T, top), dev, "weights")
    out, o_at, old = _out(out, x, T, w.hidden, dev, given)
    need = _bytes(E.MOE_UP | E.MOE_DOWN | bit, T, top, w.experts, H, w.inner)
    buf, w_at = _room(workspace, x, need, dev, raw, given)
    rc = getattr(_lib(), call)(T, top, w.experts, H, w.inner, at, ld, i_at, f_at, w.up_at, w.up_scale_at, w.down_at,
                               w.down_scale_at, o_at, old, w_at, need, _status(status, dev), raw)
    if rc:
        E.check(rc, "experts")
    return out
