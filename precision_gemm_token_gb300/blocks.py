"""Tensor-level helpers over the C ABI's projections in 8-bit blocks (E4M3
codes, one fp32 scale per 128 elements of an activation row and per 128 x 128
block of a weight): check what the library cannot see, allocate outputs with
torch on the launching stream, call the binding, raise on a non-OK status. No
arithmetic of the operators happens here.

    w = quantize_weight(W_bf16)                        # once, at load time; or BlockWeight(codes, scale)
    ws = BlockWorkspace(device)                        # one for all layers (and for the calls of `moe`)
    y = block_linear(x, w, workspace=ws)               # bf16 [M, K] -> bf16 [M, N]
    xq, xs = block_quant(x)                            # the two halves of it, where several
    y = block_matmul(xq, xs, w)                        # projections share their input
"""
from __future__ import annotations

from functools import lru_cache
from typing import Optional

import torch

from . import _binding as E

BLOCK = 128
_BF16, _F32, _U8, _I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
_lib = E.load


def _bad(what):
    raise E.EpiloraError(E.EPILORA_ERR_INVALID_ARG, what)


def _blocks(n):
    return -(-n // BLOCK)


def _start(t, stream):
    """(device, raw handle of the launching stream, the stream where it is
    given: what a call allocates is then made on it)"""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        _bad("tensors on the current CUDA device wanted")
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev), None
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    return dev, stream.cuda_stream, stream


def _new(like, shape, dtype, stream):
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _matrix(t, dtype, dev, what, rows=None, cols=None):
    """(address, rows, columns, row stride) of a matrix with contiguous rows."""
    if t.dtype is not dtype or t.dim() != 2 or t.get_device() != dev:
        _bad(f"{what}: {dtype} matrix on device {dev} wanted")
    m, n = t.shape
    if (rows is not None and m != rows) or (cols is not None and n != cols):
        _bad(f"{what}: [{'any' if rows is None else rows}, {'any' if cols is None else cols}] wanted, not [{m}, {n}]")
    ld, es = t.stride()
    if (es != 1 and n > 1) or (ld < n and m > 1):
        _bad(what + ": contiguous rows wanted")
    return t.data_ptr(), m, n, (ld if m > 1 else -(-n // 8) * 8)


def _array(t, dtype, shape, dev, what):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        _bad(f"{what}: contiguous {dtype} {list(shape)} on device {dev} wanted")
    return t.data_ptr()


def _made(t, like, shape, dtype, dev, stream, what):
    """(an output, its address): the caller's, or a new one."""
    if t is None:
        t = _new(like, shape, dtype, stream)
        return t, t.data_ptr()
    return t, _array(t, dtype, shape, dev, what)


# bytes of workspace, asked of the library once per shape
_linear_bytes = lru_cache(1024)(E.epilora_block_linear_workspace_bytes)


def _status(status, dev):
    if status is None:
        return None
    if status.dtype is not _I32 or status.numel() < 1 or status.get_device() != dev:
        _bad("status: int32 on the tensors' device wanted")
    return status.data_ptr()


class BlockWeight:
    """E4M3 codes uint8 [N, K] and fp32 scales [ceil(N / 128), ceil(K / 128)]
    of their 128 x 128 blocks. The tensors stay the caller's."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor):
        if codes.dtype is not _U8 or codes.dim() != 2 or not codes.is_contiguous():
            _bad("weight codes: contiguous uint8 [N, K] wanted")
        self.N, self.K = codes.shape
        self.dev = codes.get_device()
        self.scale_at = _array(scale, _F32, (_blocks(self.N), _blocks(self.K)), self.dev, "weight scales")
        self.codes, self.scale = codes, scale
        self.codes_at = codes.data_ptr()


class BlockWorkspace:
    """Caller-owned workspace of block_linear and of the calls of `moe`, grown
    on demand; nothing in it has to be initialized. Calls that share one have
    to be ordered on one stream, and a captured graph wants it kept as long as
    the graph: a buffer that a capture has used is kept when a larger one
    takes its place, and so is one used on a stream that torch does not own.
    `device` without an index is the current one at this
    point."""

    def __init__(self, device):
        device = torch.device(device)
        if device.type != "cuda":
            _bad(f"workspace: a CUDA device wanted, not {device}")
        self.device = torch.device("cuda", torch.cuda.current_device()) if device.index is None else device
        self._buf, self._captured, self._kept = None, False, []
        self._own, self._foreign = None, False      # the buffer's stream; used on one that the allocator cannot know
        self._known = set()         # raw handles of the streams that the allocator knows the buffer's use on

    def get(self, need, dev, raw, stream):
        """(the buffer, its address) with room for `need` bytes, for a call on
        device `dev` and the stream of handle `raw` (`stream`: where that is
        not the current one)."""
        if self.device.index != dev:
            _bad(f"workspace: on {self.device}, the tensors on device {dev}")
        if self._buf is None or self._buf.numel() < need:
            if self._captured or self._foreign:
                self._kept.append(self._buf)
            self._buf, self._captured, self._known = None, False, set()
            self._own, self._foreign = raw, False
            if stream is None:
                self._buf = torch.empty(max(need, 1 << 20), dtype=_U8, device=self.device)
            else:
                with torch.cuda.stream(stream):
                    self._buf = torch.empty(max(need, 1 << 20), dtype=_U8, device=self.device)
            if not isinstance(stream, torch.cuda.ExternalStream):
                self._known.add(raw)
        if raw not in self._known or not self._captured:
            self._note(raw, stream)
        return self._buf, self._buf.data_ptr()

    def _note(self, raw, stream):
        """The allocator lets no other tensor have the buffer before a stream
        was used on is done with it, should the workspace be dropped or
        grow. A stream that torch does not own may be gone by then: there a
        buffer that grew is kept, and the workspace is the caller's to keep."""
        if torch.cuda.is_current_stream_capturing() if stream is None else _capturing(stream):
            self._captured = True
        elif isinstance(stream, torch.cuda.ExternalStream):
            self._foreign |= raw != self._own
        elif raw not in self._known:
            self._buf.record_stream(torch.cuda.current_stream() if stream is None else stream)
            self._known.add(raw)


def _capturing(stream):
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _room(workspace, like, need, dev, raw, stream):
    """(a tensor to keep until the call is enqueued, its address) of a call's workspace."""
    if workspace is None:
        buf = _new(like, max(need, 256), _U8, stream)
        return buf, buf.data_ptr()
    return workspace.get(need, dev, raw, stream)


def block_quant(x, codes=None, scale=None, stream=None):
    """bf16 x [M, K] -> (codes uint8 [M, K], scale fp32 [ceil(K / 128), M]),
    or into the given ones."""
    dev, raw, given = _start(x, stream)
    at, M, K, ld = _matrix(x, _BF16, dev, "x")
    codes, c_at = _made(codes, x, (M, K), _U8, dev, given, "codes")
    scale, s_at = _made(scale, x, (-(-K // BLOCK), M), _F32, dev, given, "scale")
    rc = _lib().epilora_block_quant(at, M, K, ld, c_at, s_at, M, raw)
    if rc:
        E.check(rc, "block_quant")
    return codes, scale


def quantize_weight(W, stream=None) -> BlockWeight:
    """Load-time quantization of a bf16 weight [N, K]."""
    dev, raw, given = _start(W, stream)
    at, N, K, ld = _matrix(W, _BF16, dev, "W")
    codes, scale = _new(W, (N, K), _U8, given), _new(W, (_blocks(N), _blocks(K)), _F32, given)
    _quantize_weight(at, N, K, ld, codes, scale, raw)
    return BlockWeight(codes, scale)


def _quantize_weight(at, N, K, ld, codes, scale, raw):
    rc = _lib().epilora_block_quant_weight(at, N, K, ld, codes.data_ptr(), scale.data_ptr(), raw)
    if rc:
        E.check(rc, "quantize_weight")


def _out(out, like, M, N, dev, stream):
    if out is None:
        out = _new(like, (M, N), _BF16, stream)
        return out, out.data_ptr(), N
    at, _, _, ld = _matrix(out, _BF16, dev, "out", M, N)
    return out, at, max(ld, N)


def block_matmul(codes, scale, w: BlockWeight, out=None, status=None, stream=None):
    """Product of quantized rows (codes [M, K], scale [ceil(K / 128), M]) with
    the weight: bf16 [M, N]."""
    dev, raw, given = _start(codes, stream)
    if codes.dim() != 2 or codes.shape[1] != w.K or w.dev != dev:
        _bad("block_matmul: codes and the weight disagree in K or device")
    M = codes.shape[0]
    c_at = _array(codes, _U8, (M, w.K), dev, "codes")
    s_at = _array(scale, _F32, (_blocks(w.K), M), dev, "scale")
    out, o_at, ld = _out(out, codes, M, w.N, dev, given)
    rc = _lib().epilora_block_matmul(M, w.N, w.K, c_at, s_at, M, w.codes_at, w.scale_at, o_at, ld, _status(status, dev),
                                     raw)
    if rc:
        E.check(rc, "block_matmul")
    return out


def block_linear(x, w: BlockWeight, out=None, workspace: Optional[BlockWorkspace] = None, status=None, stream=None):
    """bf16 x [M, K] times the weight, x quantized on the way: bf16 [M, N]."""
    dev, raw, given = _start(x, stream)
    if w.dev != dev:
        _bad("block_linear: x and the weight on different devices")
    at, M, K, ld = _matrix(x, _BF16, dev, "x", None, w.K)
    out, o_at, old = _out(out, x, M, w.N, dev, given)
    need = _linear_bytes(M, K)
    buf, w_at = _room(workspace, x, need, dev, raw, given)
    rc = _lib().epilora_block_linear(M, w.N, K, at, ld, w.codes_at, w.scale_at, o_at, old, w_at, need,
                                     _status(status, dev), raw)
    if rc:
        E.check(rc, "block_linear")
    return out
