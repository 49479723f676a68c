"""Tensor-level helpers over the attention entry points of the C ABI: check
what the library cannot see (types, shapes, devices), allocate outputs with
torch on the launching stream, call the binding, raise on a non-OK status. No
arithmetic of the operators happens here.

    cache = PagedKVCache(k_pages, v_pages)                 # once per layer
    ws = AttentionWorkspace(device)                        # once per model
    q = kv_append(q, k, v, cache, q_start, kv_len, page_table, cos_sin)
    o = paged_attention(q, cache, q_start, kv_len, page_table, max_new=1, workspace=ws)
    o = prompt_attention(q, k, v, q_start, workspace=ws)   # whole prompts, no cache

`q`, `k`, `v` are bf16 [tokens, heads, head_dim] with any token and head
strides (slices of a fused projection's output). Sequence b owns the packed
rows q_start[b] .. q_start[b+1] - 1 and holds kv_len[b] tokens with them.
"""
from __future__ import annotations

import struct
from typing import Optional

import torch

from . import _binding as E

_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
# epilora_kv_batch as bytes: a decode step calls these helpers once or twice
# per layer, and packing eight numbers costs a third of a ctypes struct
_pack_batch = struct.Struct("iiiiqPPP").pack
_lib = E.load


def _bad(what):
    raise E.EpiloraError(E.EPILORA_ERR_INVALID_ARG, what)


def _rows(t, shape, dev, what):
    """(address, token stride, head stride) of rows [tokens, heads, head_dim]
    of the given shape; a dimension of one element has no stride of its own."""
    if t.dtype is not _BF16 or t.shape != shape or t.get_device() != dev:
        _bad(f"{what}: bf16 [tokens, heads, head_dim] = {tuple(shape)} on device {dev} wanted")
    n, h, d = shape
    ts, hs, es = t.stride()
    if es != 1 and d > 1:
        _bad(what + ": the elements of a head have to be contiguous")
    if h == 1:
        hs = d
    return t.data_ptr(), (ts if n > 1 else h * hs), hs


def _index(t, n, dev, what):
    if t.dtype is not _I32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        _bad(f"{what}: contiguous int32 [{n}] on device {dev} wanted")
    return t.data_ptr()


def _start(q, stream):
    """(shape of q, its device, the raw handle of the launching stream, and
    the stream itself where it is given: what a call allocates is then made
    on it)"""
    shape = q.shape
    if len(shape) != 3:
        _bad("q: [tokens, heads, head_dim] wanted")
    dev = q.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        _bad("tensors on the current CUDA device wanted")
    if stream is None:
        return shape, dev, torch._C._cuda_getCurrentRawStream(dev), None
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    return shape, dev, stream.cuda_stream, stream


def _new(q, shape, stream):
    if stream is None:
        return torch.empty(shape, dtype=_BF16, device=q.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=_BF16, device=q.device)


def _own_workspace(q, dim):
    """A workspace of one call: only what has to be zero is filled."""
    need = E.epilora_attention_workspace_bytes(dim) or 256      # (0: a head size that the call will refuse)
    buf = torch.empty(need, dtype=_U8, device=q.device)
    buf[:E.epilora_attention_workspace_zero_bytes()].zero_()
    return buf, buf.data_ptr(), need


def _workspace(workspace, q, dim, raw, stream):
    """(tensor, address, bytes), in order on the launching stream."""
    if workspace is None:
        if stream is None:
            return _own_workspace(q, dim)
        with torch.cuda.stream(stream):
            return _own_workspace(q, dim)
    if workspace.device.index != q.get_device():
        _bad(f"workspace: on {workspace.device}, the tensors on device {q.get_device()}")
    if raw not in workspace.known:
        workspace.note(raw, stream)
    if workspace.head is None:
        buf = workspace.get(dim)
    else:
        with torch.cuda.stream(stream):
            buf = workspace.get(dim)
    return buf, buf.data_ptr(), buf.numel()


def _status(status, dev):
    if status is None:
        return None
    if status.dtype is not _I32 or status.numel() < 1 or status.get_device() != dev:
        _bad("status: int32 on the tensors' device wanted")
    return status.data_ptr()


class PagedKVCache:
    """One layer's cache: k and v [num_pages, kv_heads, page_size, head_dim],
    bf16, or uint8 E4M3 codes with k_scale / v_scale fp32 [kv_heads]. Any
    strides with contiguous elements per head: a pool stored
    [num_pages, page_size, kv_heads, head_dim] is passed as
    pool.transpose(1, 2). The tensors stay the caller's."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if not (k.dim() == 4 and k.shape == v.shape and k.dtype is v.dtype and k.dtype in (_BF16, _U8)):
            _bad("cache: two bf16 or uint8 [num_pages, kv_heads, page_size, head_dim] wanted")
        e4m3 = k.dtype is _U8
        if not ((k_scale is not None and v_scale is not None) if e4m3 else (k_scale is None and v_scale is None)):
            _bad("cache: scales go with E4M3 codes, and only with them")
        for s in (k_scale, v_scale):
            if not (s is None or (s.dtype is _F32 and s.shape == k.shape[1:2] and s.is_contiguous())):
                _bad("cache: scales are contiguous fp32 [kv_heads]")
        if any(t is not None and t.get_device() != k.get_device() for t in (v, k_scale, v_scale)):
            _bad("cache: tensors on different devices")
        pages, heads, size, dim = k.shape
        c = E.KvCache(kv_fmt=E.KV_E4M3 if e4m3 else E.KV_BF16, kv_heads=heads, head_dim=dim, page_size=size,
                      num_pages=pages, reserved=0, k=k.data_ptr(), v=v.data_ptr(),
                      k_scale=k_scale.data_ptr() if e4m3 else None, v_scale=v_scale.data_ptr() if e4m3 else None)
        for n, t in (("k", k), ("v", v)):
            s = t.stride()
            if s[3] != 1:
                _bad("cache: the elements of a head's row have to be contiguous")
            for axis, name in ((0, "page"), (1, "head"), (2, "token")):
                # a dimension of one element has no stride of its own
                setattr(c, f"{n}_{name}_stride", s[axis] if t.shape[axis] > 1 else dim)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.dev = k.get_device()
        self.device, self.kv_heads, self.head_dim, self.page_size = k.device, heads, dim, size
        self.struct = c
        self.address = E.ctypes.addressof(c)


class AttentionWorkspace:
    """Caller-owned workspace of the attention calls (see
    epilora_attention_workspace_bytes) for both head sizes, allocated and
    zero-filled here: every stream, and every graph whether captured before or
    after the first call, finds it ready. `device` without an index is the
    current one at this point. Calls that share one have to be ordered on one
    stream, and a captured graph wants it kept as long as the graph. After a
    call that recorded EPILORA_ERR_TIMEOUT, take a new one.

    One made while the current stream is being captured is zeroed by the graph
    only, when that is replayed; each call with it therefore zeroes the part
    that has to be zero."""

    def __init__(self, device):
        device = torch.device(device)
        if device.type != "cuda":
            _bad(f"workspace: a CUDA device wanted, not {device}")
        self.device = torch.device("cuda", torch.cuda.current_device()) if device.index is None else device
        self.head = None            # what every call has to zero
        self.known = set()          # raw handles of the streams that the allocator knows the buffer's use on
        self._buf = self._make()

    def _make(self):
        with torch.cuda.device(self.device):
            need = max(E.epilora_attention_workspace_bytes(d) for d in (64, 128))
            buf = torch.zeros(need, dtype=_U8, device=self.device)
            if torch.cuda.is_current_stream_capturing():
                self.head = buf[:E.epilora_attention_workspace_zero_bytes()]
            else:
                stream = torch.cuda.current_stream()
                stream.synchronize()
                self.known.add(stream.cuda_stream)
        return buf

    def get(self, head_dim):
        """The buffer, ready for a call on the current stream."""
        if self.head is not None:
            self.head.zero_()
        return self._buf

    def note(self, raw, stream):
        """The first call on `stream` (None: the current one; `raw` its
        handle): the allocator will let no other tensor have the buffer before
        that stream is done with it, should the workspace be dropped. A stream
        that torch does not own may be gone by then: there it is the caller's
        to keep the workspace."""
        if isinstance(stream, torch.cuda.ExternalStream):
            return
        if stream is None:
            stream = torch.cuda.current_stream()
        if not torch.cuda.is_current_stream_capturing():
            self._buf.record_stream(stream)
            self.known.add(raw)


def _batch(tokens, q_start, kv_len, page_table, max_new, dev):
    """epilora_kv_batch (as bytes)."""
    n = q_start.numel() - 1
    if n < 0:
        _bad("q_start: [sequences + 1] wanted")
    starts, lens = _index(q_start, n + 1, dev, "q_start"), _index(kv_len, n, dev, "kv_len")
    if page_table.dtype is not _I32 or page_table.dim() != 2 or page_table.get_device() != dev:
        _bad(f"page_table: int32 [{n}, pages] on device {dev} wanted")
    rows, pages = page_table.shape
    ts, cs = page_table.stride()
    if rows != n or (cs != 1 and pages > 1) or (ts < pages and n > 1):
        _bad(f"page_table: [{n}, pages] with contiguous rows wanted")
    return _pack_batch(n, tokens, tokens if max_new is None else max_new, pages, ts if n > 1 else pages, starts, lens,
                       page_table.data_ptr())


def kv_append(q, k, v, cache: PagedKVCache, q_start, kv_len, page_table, cos_sin=None, interleaved=False, q_out=None,
              status=None, stream=None):
    """Append k and v [tokens, kv_heads, head_dim] to the cache, rotating q
    and k by position with cos_sin fp32 [positions, rot_dim] (cosines, then
    sines; None: no rotation). Returns the rotated q (q_out, which may be q
    itself). epilora_kv_append has the details."""
    shape, dev, raw, given = _start(q, stream)
    T, heads, dim = shape
    q_at, qt, qh = _rows(q, shape, dev, "q")
    if dim != cache.head_dim or cache.dev != dev:
        _bad("kv_append: q and the cache disagree in head_dim or device")
    kv = (T, cache.kv_heads, dim)
    k_at, kt, kh = _rows(k, kv, dev, "k")
    v_at, vt, vh = _rows(v, kv, dev, "v")
    n_pos = rot = 0
    table = None
    if cos_sin is not None:
        if cos_sin.dtype is not _F32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous() or cos_sin.get_device() != dev:
            _bad("cos_sin: contiguous fp32 [positions, rot_dim] wanted")
        n_pos, rot = cos_sin.shape
        if cos_sin.numel() == 0 and T > 0:      # (without an address it would stand for no rotation)
            _bad("cos_sin: no position or no element to rotate in it")
        table = cos_sin.data_ptr()
    batch = _batch(T, q_start, kv_len, page_table, None, dev)
    if q_out is None:
        q_out = _new(q, shape, given)
    o_at, ot, oh = _rows(q_out, shape, dev, "q_out")
    rc = _lib().epilora_kv_append(cache.address, batch, heads, q_at, qt, qh, k_at, kt, kh, v_at, vt, vh, table, n_pos,
                                  rot, 1 if interleaved else 0, o_at, ot, oh, _status(status, dev), raw)
    if rc:
        E.check(rc, "kv_append")
    return q_out


def _lse(lse, shape, dev):
    if lse is None:
        return None
    if lse.dtype is not _F32 or lse.shape != shape[:2] or not lse.is_contiguous() or lse.get_device() != dev:
        _bad("lse: contiguous fp32 [tokens, heads] wanted")
    return lse.data_ptr()


def paged_attention(q, cache: PagedKVCache, q_start, kv_len, page_table, max_new: Optional[int] = None,
                    scale: Optional[float] = None, out=None, lse=None, workspace: Optional[AttentionWorkspace] = None,
                    status=None, stream=None):
    """Attention of the new tokens q [tokens, heads, head_dim] over the cache
    (their keys and values appended before). max_new: an upper bound of the
    new tokens of any sequence, known on the host (default: all of them; 1
    for a decode step). scale defaults to head_dim ** -0.5. lse (optional,
    fp32 [tokens, heads]) receives the log of the softmax sums."""
    shape, dev, raw, given = _start(q, stream)
    T, heads, dim = shape
    q_at, qt, qh = _rows(q, shape, dev, "q")
    if dim != cache.head_dim or cache.dev != dev:
        _bad("paged_attention: q and the cache disagree in head_dim or device")
    batch = _batch(T, q_start, kv_len, page_table, max_new, dev)
    if out is None:
        out = _new(q, shape, given)
    o_at, ot, oh = _rows(out, shape, dev, "out")
    buf, w_at, w_bytes = _workspace(workspace, q, dim, raw, given)
    rc = _lib().epilora_paged_attention(cache.address, batch, heads, q_at, qt, qh, dim ** -0.5 if scale is None else scale,
                                        o_at, ot, oh, _lse(lse, shape, dev), w_at, w_bytes, _status(status, dev), raw)
    if rc:
        E.check(rc, "paged_attention")
    return out


def prompt_attention(q, k, v, q_start, scale: Optional[float] = None, out=None, lse=None,
                     workspace: Optional[AttentionWorkspace] = None, status=None, stream=None):
    """Causal attention of whole packed prompts: prompt b is the rows
    q_start[b] .. q_start[b+1] - 1 of q [tokens, heads, head_dim] and of k, v
    [tokens, kv_heads, head_dim]. Other arguments as paged_attention."""
    shape, dev, raw, given = _start(q, stream)
    T, heads, dim = shape
    q_at, qt, qh = _rows(q, shape, dev, "q")
    if k.dim() != 3:
        _bad("k: [tokens, kv_heads, head_dim] wanted")
    kv_heads = k.shape[1]
    kv = (T, kv_heads, dim)
    k_at, kt, kh = _rows(k, kv, dev, "k")
    v_at, vt, vh = _rows(v, kv, dev, "v")
    n = q_start.numel() - 1
    if n < 0:
        _bad("q_start: [sequences + 1] wanted")
    starts = _index(q_start, n + 1, dev, "q_start")
    if out is None:
        out = _new(q, shape, given)
    o_at, ot, oh = _rows(out, shape, dev, "out")
    buf, w_at, w_bytes = _workspace(workspace, q, dim, raw, given)
    rc = _lib().epilora_prompt_attention(n, T, starts, heads, kv_heads, dim, q_at, qt, qh, k_at, kt, kh, v_at, vt, vh,
                                         dim ** -0.5 if scale is None else scale, o_at, ot, oh,
                                         _lse(lse, shape, dev), w_at, w_bytes, _status(status, dev), raw)
    if rc:
        E.check(rc, "prompt_attention")
    return out
