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

import contextlib
from typing import Optional

import torch

from . import _binding as E

_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


def _want(ok, what):
    if not ok:
        raise E.EpiloraError(E.EPILORA_ERR_INVALID_ARG, what)


def _strides(t, what):
    """(token, head) strides of rows [tokens, heads, head_dim]; a dimension of
    one element has no stride of its own."""
    _want(t.dim() == 3 and t.dtype is _BF16, f"{what}: bf16 [tokens, heads, head_dim] wanted")
    n, h, d = t.shape
    s = t.stride()
    _want(s[2] == 1, f"{what}: the elements of a head have to be contiguous")
    hs = s[1] if h > 1 else d
    return (s[0] if n > 1 else h * hs), hs


def _on(device, what, *tensors):
    for t in tensors:
        _want(t is None or t.device == device, f"{what}: tensors on different devices")


def _index(t, shape, what):
    _want(t.dtype is _I32 and t.shape == shape and t.is_contiguous(), f"{what}: contiguous int32 {tuple(shape)} wanted")
    return t


def _launch(device, stream):
    """(context that allocates on the launching stream, its raw handle)"""
    _want(device.type == "cuda", "a CUDA device is wanted")
    _want(device.index == torch.cuda.current_device(), "the tensors are not on the current device")
    if stream is None:
        return contextlib.nullcontext(), torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream), stream.cuda_stream


class PagedKVCache:
    """One layer's cache: k and v [num_pages, kv_heads, page_size, head_dim],
    bf16, or uint8 E4M3 codes with k_scale / v_scale fp32 [kv_heads]. Any
    strides with contiguous elements per head: a pool stored
    [num_pages, page_size, kv_heads, head_dim] is passed as
    pool.transpose(1, 2). The tensors stay the caller's."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        _want(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.dtype in (_BF16, torch.uint8),
              "cache: two bf16 or uint8 [num_pages, kv_heads, page_size, head_dim] wanted")
        e4m3 = k.dtype is torch.uint8
        _want((k_scale is not None and v_scale is not None) if e4m3 else (k_scale is None and v_scale is None),
              "cache: scales go with E4M3 codes, and only with them")
        for s in (k_scale, v_scale):
            _want(s is None or (s.dtype is _F32 and s.shape == k.shape[1:2] and s.is_contiguous()),
                  "cache: scales are contiguous fp32 [kv_heads]")
        _on(k.device, "cache", v, k_scale, v_scale)
        pages, heads, size, dim = k.shape
        c = E.KvCache(kv_fmt=E.KV_E4M3 if e4m3 else E.KV_BF16, kv_heads=heads, head_dim=dim, page_size=size,
                      num_pages=pages, reserved=0, k=k.data_ptr(), v=v.data_ptr(),
                      k_scale=k_scale.data_ptr() if e4m3 else None, v_scale=v_scale.data_ptr() if e4m3 else None)
        for n, t in (("k", k), ("v", v)):
            s = t.stride()
            _want(s[3] == 1, "cache: the elements of a head's row have to be contiguous")
            for axis, name in ((0, "page"), (1, "head"), (2, "token")):
                # a dimension of one element has no stride of its own
                setattr(c, f"{n}_{name}_stride", s[axis] if t.shape[axis] > 1 else dim)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.kv_heads, self.head_dim, self.page_size = k.device, heads, dim, size
        self.struct = c


class AttentionWorkspace:
    """Caller-owned workspace of the attention calls (see
    epilora_attention_workspace_bytes), zero-filled when first used. Calls
    that share one have to be ordered on one stream."""

    def __init__(self, device):
        self.device = torch.device(device)
        self._buf = {}

    def get(self, head_dim):
        buf = self._buf.get(head_dim)
        if buf is None:
            need = E.epilora_attention_workspace_bytes(head_dim)
            buf = self._buf[head_dim] = torch.zeros(max(need, 256), dtype=torch.uint8, device=self.device)
        return buf


def _batch(tokens, q_start, kv_len, page_table, max_new):
    n = q_start.numel() - 1
    _want(n >= 0, "q_start: [sequences + 1] wanted")
    _index(q_start, (n + 1,), "q_start")
    _index(kv_len, (n,), "kv_len")
    _want(page_table.dtype is _I32 and page_table.dim() == 2 and page_table.shape[0] == n,
          f"page_table: int32 [{n}, pages] wanted")
    pages = page_table.shape[1]
    ts, cs = page_table.stride()
    _want((cs == 1 or pages <= 1) and (ts >= pages or n <= 1), "page_table: rows have to be contiguous")
    return E.KvBatch(n, tokens, tokens if max_new is None else max_new, pages, ts if n > 1 else pages,
                     q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr())


def kv_append(q, k, v, cache: PagedKVCache, q_start, kv_len, page_table, cos_sin=None, interleaved=False, q_out=None,
              status=None, stream=None):
    """Append k and v [tokens, kv_heads, head_dim] to the cache, rotating q
    and k by position with cos_sin fp32 [positions, rot_dim] (cosines, then
    sines; None: no rotation). Returns the rotated q (q_out, which may be q
    itself). epilora_kv_append has the details."""
    T, heads, dim = q.shape
    qs, ks, vs = _strides(q, "q"), _strides(k, "k"), _strides(v, "v")
    _want(k.shape == v.shape == (T, cache.kv_heads, dim) and dim == cache.head_dim,
          "kv_append: q, k, v and the cache disagree in shape")
    _on(cache.device, "kv_append", q, k, v, q_start, kv_len, page_table, cos_sin, q_out)
    n_pos = rot = 0
    if cos_sin is not None:
        _want(cos_sin.dtype is _F32 and cos_sin.dim() == 2 and cos_sin.is_contiguous(),
              "cos_sin: contiguous fp32 [positions, rot_dim] wanted")
        n_pos, rot = cos_sin.shape
    ctx, raw = _launch(cache.device, stream)
    batch = _batch(T, q_start, kv_len, page_table, None)
    if q_out is None:
        with ctx:
            q_out = torch.empty((T, heads, dim), dtype=_BF16, device=q.device)
    _want(q_out.shape == q.shape, "kv_append: q_out has another shape than q")
    E.check(E.epilora_kv_append(cache.struct, batch, heads, q, qs, k, ks, v, vs, cos_sin, n_pos, rot, interleaved,
                                q_out, _strides(q_out, "q_out"), status, raw), "kv_append")
    return q_out


def _outputs(q, out, lse):
    T, heads, dim = q.shape
    if out is None:
        out = torch.empty((T, heads, dim), dtype=_BF16, device=q.device)
    _want(out.shape == q.shape, "out has another shape than q")
    _want(lse is None or (lse.dtype is _F32 and lse.shape == (T, heads) and lse.is_contiguous()),
          f"lse: contiguous fp32 {(T, heads)} wanted")
    return out


def paged_attention(q, cache: PagedKVCache, q_start, kv_len, page_table, max_new: Optional[int] = None,
                    scale: Optional[float] = None, out=None, lse=None, workspace: Optional[AttentionWorkspace] = None,
                    status=None, stream=None):
    """Attention of the new tokens q [tokens, heads, head_dim] over the cache
    (their keys and values appended before). max_new: an upper bound of the
    new tokens of any sequence, known on the host (default: all of them; 1
    for a decode step). scale defaults to head_dim ** -0.5. lse (optional,
    fp32 [tokens, heads]) receives the log of the softmax sums."""
    T, heads, dim = q.shape
    qs = _strides(q, "q")
    _want(dim == cache.head_dim, "paged_attention: q and the cache disagree in head_dim")
    _on(cache.device, "paged_attention", q, q_start, kv_len, page_table, out, lse)
    ctx, raw = _launch(cache.device, stream)
    batch = _batch(T, q_start, kv_len, page_table, max_new)
    with ctx:
        out = _outputs(q, out, lse)
        ws = (workspace or AttentionWorkspace(q.device)).get(dim)
    E.check(E.epilora_paged_attention(cache.struct, batch, heads, q, qs, dim ** -0.5 if scale is None else scale, out,
                                      _strides(out, "out"), lse, ws, ws.numel(), status, raw), "paged_attention")
    return out


def prompt_attention(q, k, v, q_start, scale: Optional[float] = None, out=None, lse=None,
                     workspace: Optional[AttentionWorkspace] = None, status=None, stream=None):
    """Causal attention of whole packed prompts: prompt b is the rows
    q_start[b] .. q_start[b+1] - 1 of q [tokens, heads, head_dim] and of k, v
    [tokens, kv_heads, head_dim]. Other arguments as paged_attention."""
    T, heads, dim = q.shape
    qs, ks, vs = _strides(q, "q"), _strides(k, "k"), _strides(v, "v")
    _want(k.shape == v.shape and k.shape[0] == T and k.shape[2] == dim, "prompt_attention: q, k and v disagree in shape")
    _on(q.device, "prompt_attention", k, v, q_start, out, lse)
    n = q_start.numel() - 1
    _want(n >= 0, "q_start: [sequences + 1] wanted")
    _index(q_start, (n + 1,), "q_start")
    ctx, raw = _launch(q.device, stream)
    with ctx:
        out = _outputs(q, out, lse)
        ws = (workspace or AttentionWorkspace(q.device)).get(dim)
    E.check(E.epilora_prompt_attention(n, T, q_start, heads, k.shape[1], dim, q, qs, k, ks, v, vs,
                                       dim ** -0.5 if scale is None else scale, out, _strides(out, "out"), lse, ws,
                                       ws.numel(), status, raw), "prompt_attention")
    return out
