"""ctypes binding of libepilora.so: the C ABI of include/epilora.h, same names.

Argument marshalling only. Every data argument may be a torch tensor (its
data_ptr() is passed), a raw integer device address, or None (NULL). `stream`
may be a torch.cuda.Stream, a raw cudaStream_t integer, or None for torch's
current stream on the current device. Each function returns the library's
int status; `check()` turns a non-zero status into an exception.

There is no fallback: if the library has not been built, loading raises.
"""
from __future__ import annotations

import ctypes
import os

from .build import LIB_PATH

EPILORA_OK = 0
EPILORA_ERR_INVALID_ARG = -1
EPILORA_ERR_UNSUPPORTED = -2
EPILORA_ERR_CUDA = -3
EPILORA_ERR_TIMEOUT = -4
EPILORA_ERR_WORKSPACE = -5
FMT_FP8 = 0
FMT_NVFP4 = 1

WORKSPACE_SYNC_BYTES = 2360576      # EPILORA_WORKSPACE_SYNC_BYTES

KV_BF16 = 0
KV_E4M3 = 1

LOGITS_F32 = 0
LOGITS_BF16 = 1
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
MOE_UP = 1
MOE_DOWN = 2
MOE_F32_PARTS = 4
BLOCK_MAX_SIZE = 0x7FFF0000         # EPILORA_BLOCK_MAX_SIZE
MOE_MAX_EXPERTS = 1024              # EPILORA_MOE_MAX_EXPERTS
MOE_MAX_TOP = 32                    # EPILORA_MOE_MAX_TOP

_c_int, _vp, _sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
_i64, _f32 = ctypes.c_int64, ctypes.c_float


class KvCache(ctypes.Structure):
    """epilora_kv_cache"""
    _fields_ = [("kv_fmt", _c_int), ("kv_heads", _c_int), ("head_dim", _c_int), ("page_size", _c_int),
                ("num_pages", _c_int), ("reserved", _c_int), ("k", _vp), ("v", _vp),
                ("k_page_stride", _i64), ("k_head_stride", _i64), ("k_token_stride", _i64),
                ("v_page_stride", _i64), ("v_head_stride", _i64), ("v_token_stride", _i64),
                ("k_scale", _vp), ("v_scale", _vp)]


class KvBatch(ctypes.Structure):
    """epilora_kv_batch"""
    _fields_ = [("n_seqs", _c_int), ("n_tokens", _c_int), ("max_new", _c_int), ("table_pages", _c_int),
                ("table_stride", _i64), ("q_start", _vp), ("kv_len", _vp), ("page_table", _vp)]


# name -> (restype, argtypes), in the order of include/epilora.h
SIGNATURES = {
    "epilora_abi_version": (_c_int, []),
    "epilora_status_string": (ctypes.c_char_p, [_c_int]),
    "epilora_quant_act": (_c_int, [_c_int, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "epilora_nvfp4_global_scale": (_c_int, [_vp, _sz, _vp, _vp]),
    "epilora_lora_shrink": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp]),
    "epilora_gemm_lora_epilogue": (_c_int, [_c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                            _vp, _vp, _c_int, _c_int, _vp, _vp, _vp, _c_int, _c_int, _vp, _vp]),
    "epilora_workspace_bytes": (_sz, [_c_int, _c_int, _c_int, _c_int]),
    "epilora_layer_workspace_bytes": (_sz, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "epilora_layer_forward_kernels": (_c_int, [_c_int, _c_int, _c_int, _c_int]),
    "epilora_test_drop_shrink_results": (_c_int, [_c_int]),
    "epilora_set_decode_path": (_c_int, [_c_int]),
    "epilora_layer_forward": (_c_int, [_c_int, _c_int, _c_int, _c_int, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _vp, _c_int, _c_int, _vp, _vp, _vp, _c_int, _vp, _sz, _vp, _vp]),
    "epilora_layer_forward_fp8_adapters": (_c_int, [_c_int, _c_int, _c_int, _c_int, _vp, _c_int, _vp, _vp, _vp, _vp,
                                                    _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _vp, _vp, _vp, _c_int,
                                                    _vp, _sz, _vp, _vp]),
    "epilora_layer_forward_noalloc": (_c_int, [_c_int, _c_int, _c_int, _c_int, _vp, _c_int, _vp, _vp, _vp, _vp,
                                               _vp, _vp, _vp, _c_int, _c_int, _vp, _vp, _vp, _c_int, _vp, _vp]),
    "epilora_layer_forward_slices": (_c_int, [_c_int, _c_int, _c_int, _c_int, _vp, _c_int, _vp, _vp, _vp, _vp, _vp,
                                              _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_int, _vp,
                                              _sz, _vp, _vp]),
    "epilora_kv_append": (_c_int, [_vp, _vp, _c_int, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _c_int,
                                   _c_int, _c_int, _vp, _i64, _i64, _vp, _vp]),
    "epilora_attention_workspace_bytes": (_sz, [_c_int]),
    "epilora_attention_workspace_zero_bytes": (_sz, []),
    "epilora_paged_attention": (_c_int, [_vp, _vp, _c_int, _vp, _i64, _i64, _f32, _vp, _i64, _i64, _vp, _vp, _sz, _vp,
                                         _vp]),
    "epilora_prompt_attention": (_c_int, [_c_int, _c_int, _vp, _c_int, _c_int, _c_int, _vp, _i64, _i64, _vp, _i64,
                                          _i64, _vp, _i64, _i64, _f32, _vp, _i64, _i64, _vp, _vp, _sz, _vp, _vp]),
    "epilora_block_quant": (_c_int, [_vp, _c_int, _c_int, _i64, _vp, _vp, _i64, _vp]),
    "epilora_block_quant_weight": (_c_int, [_vp, _c_int, _c_int, _i64, _vp, _vp, _vp]),
    "epilora_block_matmul": (_c_int, [_c_int, _c_int, _c_int, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp]),
    "epilora_test_late_block_copies": (_c_int, [_c_int]),
    "epilora_block_linear_workspace_bytes": (_sz, [_c_int, _c_int]),
    "epilora_block_linear": (_c_int, [_c_int, _c_int, _c_int, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _sz, _vp, _vp]),
    "epilora_moe_route": (_c_int, [_c_int, _c_int, _c_int, _vp, _c_int, _i64, _vp, _c_int, _c_int, _c_int, _c_int,
                                   _c_int, _f32, _vp, _vp, _vp]),
    "epilora_moe_workspace_bytes": (_sz, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "epilora_moe_experts_up": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                        _vp, _sz, _vp, _vp]),
    "epilora_moe_experts_down": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                          _i64, _vp, _sz, _vp, _vp]),
    "epilora_moe_experts": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _vp, _i64, _vp, _sz, _vp, _vp]),
    "epilora_moe_experts_down_f32": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp,
                                              _vp, _i64, _vp, _sz, _vp, _vp]),
    "epilora_moe_experts_f32": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                         _vp, _vp, _i64, _vp, _sz, _vp, _vp]),
}

_lib = None


class EpiloraError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_name(status)} ({status})" if what else f"{status_name(status)} ({status})")


def load(path: str | None = None):
    """Load libepilora.so (built in-tree by precision_gemm_token_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libepilora.so is not built ({path}); run precision_gemm_token_gb300.build.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _p(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def status_name(status: int) -> str:
    try:
        return load().epilora_status_string(int(status)).decode()
    except Exception:  # library missing: still name the code
        return {0: "EPILORA_OK", -1: "EPILORA_ERR_INVALID_ARG", -2: "EPILORA_ERR_UNSUPPORTED",
                -3: "EPILORA_ERR_CUDA", -4: "EPILORA_ERR_TIMEOUT", -5: "EPILORA_ERR_WORKSPACE"}.get(status, "?")


def check(status: int, what: str = "") -> None:
    if status != EPILORA_OK:
        raise EpiloraError(status, what)


def epilora_abi_version() -> int:
    return load().epilora_abi_version()


def epilora_status_string(status: int) -> str:
    return load().epilora_status_string(int(status)).decode()


def epilora_quant_act(fmt, X, M, K, ldx, Xq, x_scale, x_block_scale, x_global_scale, status_dev=None,
                      stream=None) -> int:
    return load().epilora_quant_act(fmt, _p(X), M, K, ldx, _p(Xq), _p(x_scale), _p(x_block_scale),
                                    _p(x_global_scale), _p(status_dev), _stream(stream))


def epilora_nvfp4_global_scale(T, n, g_out, stream=None) -> int:
    return load().epilora_nvfp4_global_scale(_p(T), n, _p(g_out), _stream(stream))


def epilora_lora_shrink(X, M, K, ldx, A, L, r, idx, mask, S, status_dev=None, stream=None) -> int:
    return load().epilora_lora_shrink(_p(X), M, K, ldx, _p(A), L, r, _p(idx), _p(mask), _p(S), _p(status_dev),
                                      _stream(stream))


def epilora_gemm_lora_epilogue(fmt, M, N, K, Xq, x_scale, x_block_scale, x_global_scale, Wq, w_scale,
                               w_block_scale, w_global_scale, S, B, L, r, idx, mask, Y, ldy, pdl_dependent=0,
                               status_dev=None, stream=None) -> int:
    return load().epilora_gemm_lora_epilogue(fmt, M, N, K, _p(Xq), _p(x_scale), _p(x_block_scale),
                                             _p(x_global_scale), _p(Wq), _p(w_scale), _p(w_block_scale),
                                             _p(w_global_scale), _p(S), _p(B), L, r, _p(idx), _p(mask), _p(Y), ldy,
                                             int(pdl_dependent), _p(status_dev), _stream(stream))


def epilora_workspace_bytes(fmt, M, K, r) -> int:
    return load().epilora_workspace_bytes(fmt, M, K, r)


def epilora_layer_workspace_bytes(fmt, M, N, K, r) -> int:
    return load().epilora_layer_workspace_bytes(fmt, M, N, K, r)


def epilora_layer_forward_kernels(fmt, M, K, r) -> int:
    return load().epilora_layer_forward_kernels(fmt, M, K, r)


DECODE_PATH_AUTO, DECODE_PATH_SINGLE, DECODE_PATH_TWO = 0, 1, 2


def epilora_set_decode_path(policy: int) -> int:
    """Decode-path policy for later calls (DECODE_PATH_AUTO: the single kernel
    for FP8, the shrink grid and GEMM for NVFP4; _SINGLE: the single kernel
    wherever it can run; _TWO: never). Returns the previous policy."""
    rc = load().epilora_set_decode_path(policy)
    check(rc if rc < 0 else 0, "set_decode_path")
    return rc


def epilora_test_drop_shrink_results(on: bool) -> None:
    """Test hook: the single-kernel path's shrink items publish nothing
    while on (finishers then time out with EPILORA_ERR_TIMEOUT)."""
    load().epilora_test_drop_shrink_results(1 if on else 0)


def epilora_layer_forward(fmt, M, N, K, X, ldx, Wq, w_scale, w_block_scale, w_global_scale, x_global_scale, A, B,
                          L, r, idx, mask, Y, ldy, workspace, workspace_bytes, status_dev=None, stream=None) -> int:
    return load().epilora_layer_forward(fmt, M, N, K, _p(X), ldx, _p(Wq), _p(w_scale), _p(w_block_scale),
                                        _p(w_global_scale), _p(x_global_scale), _p(A), _p(B), L, r, _p(idx),
                                        _p(mask), _p(Y), ldy, _p(workspace), workspace_bytes, _p(status_dev),
                                        _stream(stream))


def epilora_layer_forward_slices(fmt, M, N, K, X, ldx, Wq, w_scale, w_block_scale, w_global_scale, x_global_scale,
                                 A, B, L, r, n_slices, slice_end, idx, mask, Y, ldy, workspace, workspace_bytes,
                                 status_dev=None, stream=None) -> int:
    """slice_end: a sequence of n_slices column ends (host ints)."""
    ends = (ctypes.c_int * max(1, n_slices))(*[int(e) for e in slice_end])
    return load().epilora_layer_forward_slices(fmt, M, N, K, _p(X), ldx, _p(Wq), _p(w_scale), _p(w_block_scale),
                                               _p(w_global_scale), _p(x_global_scale), _p(A), _p(B), L, r,
                                               n_slices, ctypes.cast(ends, ctypes.c_void_p), _p(idx), _p(mask),
                                               _p(Y), ldy, _p(workspace), workspace_bytes, _p(status_dev),
                                               _stream(stream))


def epilora_layer_forward_fp8_adapters(fmt, M, N, K, X, ldx, Wq, w_scale, w_block_scale, w_global_scale,
                                       x_global_scale, Aq, a_scale, Bq, b_scale, L, r, idx, mask, Y, ldy, workspace,
                                       workspace_bytes, status_dev=None, stream=None) -> int:
    return load().epilora_layer_forward_fp8_adapters(fmt, M, N, K, _p(X), ldx, _p(Wq), _p(w_scale), _p(w_block_scale),
                                                     _p(w_global_scale), _p(x_global_scale), _p(Aq), _p(a_scale),
                                                     _p(Bq), _p(b_scale), L, r, _p(idx), _p(mask), _p(Y), ldy,
                                                     _p(workspace), workspace_bytes, _p(status_dev), _stream(stream))


def epilora_layer_forward_noalloc(fmt, M, N, K, X, ldx, Wq, w_scale, w_block_scale, w_global_scale,
                                  x_global_scale, A, B, L, r, idx, mask, Y, ldy, status_dev=None,
                                  stream=None) -> int:
    return load().epilora_layer_forward_noalloc(fmt, M, N, K, _p(X), ldx, _p(Wq), _p(w_scale), _p(w_block_scale),
                                                _p(w_global_scale), _p(x_global_scale), _p(A), _p(B), L, r,
                                                _p(idx), _p(mask), _p(Y), ldy, _p(status_dev), _stream(stream))


def epilora_kv_append(cache: KvCache, batch: KvBatch, heads, Q, q_strides, K, k_strides, V, v_strides, cos_sin, n_pos,
                      rot_dim, interleaved, Qout, qo_strides, status_dev=None, stream=None) -> int:
    """Strides are (token, head) pairs in elements."""
    return load().epilora_kv_append(ctypes.addressof(cache), ctypes.addressof(batch), heads, _p(Q), *q_strides, _p(K),
                                    *k_strides, _p(V), *v_strides, _p(cos_sin), n_pos, rot_dim, int(interleaved),
                                    _p(Qout), *qo_strides, _p(status_dev), _stream(stream))


def epilora_attention_workspace_bytes(head_dim) -> int:
    return load().epilora_attention_workspace_bytes(head_dim)


def epilora_attention_workspace_zero_bytes() -> int:
    return load().epilora_attention_workspace_zero_bytes()


def epilora_paged_attention(cache: KvCache, batch: KvBatch, heads, Q, q_strides, scale, O, o_strides, lse, workspace,
                            workspace_bytes, status_dev=None, stream=None) -> int:
    return load().epilora_paged_attention(ctypes.addressof(cache), ctypes.addressof(batch), heads, _p(Q), *q_strides,
                                          scale, _p(O), *o_strides, _p(lse), _p(workspace), workspace_bytes,
                                          _p(status_dev), _stream(stream))


def epilora_prompt_attention(n_seqs, n_tokens, q_start, heads, kv_heads, head_dim, Q, q_strides, K, k_strides, V,
                             v_strides, scale, O, o_strides, lse, workspace, workspace_bytes, status_dev=None,
                             stream=None) -> int:
    return load().epilora_prompt_attention(n_seqs, n_tokens, _p(q_start), heads, kv_heads, head_dim, _p(Q), *q_strides,
                                           _p(K), *k_strides, _p(V), *v_strides, scale, _p(O), *o_strides, _p(lse),
                                           _p(workspace), workspace_bytes, _p(status_dev), _stream(stream))


def epilora_block_quant(X, M, K, ldx, Xq, x_scale, x_scale_ld, stream=None) -> int:
    return load().epilora_block_quant(_p(X), M, K, ldx, _p(Xq), _p(x_scale), x_scale_ld, _stream(stream))


def epilora_block_quant_weight(W, N, K, ldw, Wq, w_scale, stream=None) -> int:
    return load().epilora_block_quant_weight(_p(W), N, K, ldw, _p(Wq), _p(w_scale), _stream(stream))


def epilora_block_matmul(M, N, K, Xq, x_scale, x_scale_ld, Wq, w_scale, Y, ldy, status_dev=None, stream=None) -> int:
    return load().epilora_block_matmul(M, N, K, _p(Xq), _p(x_scale), x_scale_ld, _p(Wq), _p(w_scale), _p(Y), ldy,
                                       _p(status_dev), _stream(stream))


def epilora_test_late_block_copies(on: bool) -> None:
    """Test hook: the products in 8-bit blocks wait for bytes that nobody
    copies while on (they end with EPILORA_ERR_TIMEOUT and give NaN)."""
    load().epilora_test_late_block_copies(1 if on else 0)


def epilora_block_linear_workspace_bytes(M, K) -> int:
    return load().epilora_block_linear_workspace_bytes(M, K)


def epilora_block_linear(M, N, K, X, ldx, Wq, w_scale, Y, ldy, workspace, workspace_bytes, status_dev=None,
                         stream=None) -> int:
    return load().epilora_block_linear(M, N, K, _p(X), ldx, _p(Wq), _p(w_scale), _p(Y), ldy, _p(workspace),
                                       workspace_bytes, _p(status_dev), _stream(stream))


def epilora_moe_route(tokens, experts, top, logits, logits_fmt, ld, bias, scoring, groups, top_groups, group_best,
                      renormalize, scale, ids, weights, stream=None) -> int:
    return load().epilora_moe_route(tokens, experts, top, _p(logits), logits_fmt, ld, _p(bias), scoring, groups,
                                    top_groups, group_best, int(renormalize), scale, _p(ids), _p(weights),
                                    _stream(stream))


def epilora_moe_workspace_bytes(what, tokens, top, experts, hidden, inner) -> int:
    return load().epilora_moe_workspace_bytes(what, tokens, top, experts, hidden, inner)


def epilora_moe_experts_up(tokens, top, experts, hidden, inner, X, ldx, ids, Wup, wup_scale, Hq, h_scale, workspace,
                           workspace_bytes, status_dev=None, stream=None) -> int:
    return load().epilora_moe_experts_up(tokens, top, experts, hidden, inner, _p(X), ldx, _p(ids), _p(Wup),
                                         _p(wup_scale), _p(Hq), _p(h_scale), _p(workspace), workspace_bytes,
                                         _p(status_dev), _stream(stream))


def epilora_moe_experts_down(tokens, top, experts, hidden, inner, Hq, h_scale, ids, weights, Wdown, wdown_scale, Y, ldy,
                             workspace, workspace_bytes, status_dev=None, stream=None) -> int:
    return load().epilora_moe_experts_down(tokens, top, experts, hidden, inner, _p(Hq), _p(h_scale), _p(ids),
                                           _p(weights), _p(Wdown), _p(wdown_scale), _p(Y), ldy, _p(workspace),
                                           workspace_bytes, _p(status_dev), _stream(stream))


def epilora_moe_experts_down_f32(tokens, top, experts, hidden, inner, Hq, h_scale, ids, weights, Wdown, wdown_scale, Y,
                                 ldy, workspace, workspace_bytes, status_dev=None, stream=None) -> int:
    return load().epilora_moe_experts_down_f32(tokens, top, experts, hidden, inner, _p(Hq), _p(h_scale), _p(ids),
                                               _p(weights), _p(Wdown), _p(wdown_scale), _p(Y), ldy, _p(workspace),
                                               workspace_bytes, _p(status_dev), _stream(stream))


def epilora_moe_experts(tokens, top, experts, hidden, inner, X, ldx, ids, weights, Wup, wup_scale, Wdown, wdown_scale,
                        Y, ldy, workspace, workspace_bytes, status_dev=None, stream=None) -> int:
    return load().epilora_moe_experts(tokens, top, experts, hidden, inner, _p(X), ldx, _p(ids), _p(weights), _p(Wup),
                                      _p(wup_scale), _p(Wdown), _p(wdown_scale), _p(Y), ldy, _p(workspace),
                                      workspace_bytes, _p(status_dev), _stream(stream))


def epilora_moe_experts_f32(tokens, top, experts, hidden, inner, X, ldx, ids, weights, Wup, wup_scale, Wdown,
                            wdown_scale, Y, ldy, workspace, workspace_bytes, status_dev=None, stream=None) -> int:
    return load().epilora_moe_experts_f32(tokens, top, experts, hidden, inner, _p(X), ldx, _p(ids), _p(weights),
                                          _p(Wup), _p(wup_scale), _p(Wdown), _p(wdown_scale), _p(Y), ldy,
                                          _p(workspace), workspace_bytes, _p(status_dev), _stream(stream))
