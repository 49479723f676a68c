"""GB300 (sm_103a) multi-tenant LoRA linear layer of an LLM decode step.

    Y = bf16( dequant(Q(X) . Q(W)^T) + mask * (X . A[idx]^T) . B[idx]^T )

The computation lives in libepilora.so (hand-written CUDA: per-token FP8 /
NVFP4 quantizer, multi-adapter shrink, tcgen05 GEMM with the LoRA epilogue
launched as the shrink's programmatic dependent) behind the C ABI of
include/epilora.h. Between the qkv and o projections of a decoder layer the
library has the attention: a paged key/value cache (append with the position
rotation, attention of new tokens over it) and attention of packed prompts. For
weights in FP8 with a scale per 128 x 128 block it has the quantizer, the
projection and the layers of a mixture of experts (routing, the experts' MLPs).
This package is its ctypes binding (`_binding`, same function names as the C
ABI) plus `tensors` (the projections), `attention`, `blocks` (projections in
8-bit blocks) and `moe`, thin helpers that allocate outputs with torch and call
the binding. There is no CPU fallback.
"""
from ._binding import (  # noqa: F401
    BLOCK_MAX_SIZE,
    EPILORA_ERR_CUDA,
    EPILORA_ERR_INVALID_ARG,
    EPILORA_ERR_TIMEOUT,
    EPILORA_ERR_UNSUPPORTED,
    EPILORA_ERR_WORKSPACE,
    DECODE_PATH_AUTO,
    DECODE_PATH_SINGLE,
    DECODE_PATH_TWO,
    EPILORA_OK,
    FMT_FP8,
    FMT_NVFP4,
    KV_BF16,
    KV_E4M3,
    LOGITS_BF16,
    LOGITS_F32,
    MOE_DOWN,
    MOE_F32_PARTS,
    MOE_MAX_EXPERTS,
    MOE_MAX_TOP,
    MOE_UP,
    SCORE_SIGMOID,
    SCORE_SOFTMAX,
    WORKSPACE_SYNC_BYTES,
    EpiloraError,
    KvBatch,
    KvCache,
    check,
    epilora_abi_version,
    epilora_attention_workspace_bytes,
    epilora_attention_workspace_zero_bytes,
    epilora_block_linear,
    epilora_block_linear_workspace_bytes,
    epilora_block_matmul,
    epilora_block_quant,
    epilora_block_quant_weight,
    epilora_gemm_lora_epilogue,
    epilora_kv_append,
    epilora_layer_forward,
    epilora_layer_forward_fp8_adapters,
    epilora_layer_forward_kernels,
    epilora_test_late_block_copies,
    epilora_test_drop_shrink_results,
    epilora_layer_forward_noalloc,
    epilora_layer_forward_slices,
    epilora_layer_workspace_bytes,
    epilora_lora_shrink,
    epilora_moe_experts,
    epilora_moe_experts_down,
    epilora_moe_experts_down_f32,
    epilora_moe_experts_f32,
    epilora_moe_experts_up,
    epilora_moe_route,
    epilora_moe_workspace_bytes,
    epilora_nvfp4_global_scale,
    epilora_paged_attention,
    epilora_prompt_attention,
    epilora_quant_act,
    epilora_set_decode_path,
    epilora_status_string,
    epilora_workspace_bytes,
    load,
)
from .build import LIB_PATH, build  # noqa: F401
