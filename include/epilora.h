/*
 * epilora.h — C ABI of the multi-tenant LoRA linear layer of an LLM decode step
 * on NVIDIA GB300 (sm_103a).
 *
 *   Y[t,:] = bf16( dequant( Q(X)[t,:] . Q(W)^T ) + mask[t] * (x_t . A[idx_t]^T) . B[idx_t]^T )
 *
 * The operation is the one defined on the EpiLoRA page ("Fusing Many LoRA
 * Adapters into Low-Precision GEMMs for Serving and RL"):
 *   - §Background and motivation › The cost of the separate adapter path:
 *     shrink h = x A^T, expand h B^T added to the projection's output;
 *   - §Design › Multi-adapter kernels › K1 and K2: per-token activation
 *     quantization for the low-precision base GEMM, h from the bf16
 *     activations, the GEMM epilogue applies the scales then adds h B^T;
 *   - §Design › Multi-adapter kernels › The decode path: the shrink is
 *     launched first, the GEMM as its programmatic dependent, waiting for h
 *     only before its epilogue;
 * and on the PreFT page ("PreFT: Prefill-only finetuning for efficient
 * inference", Core claim): the adapter applies to prefill tokens only, which
 * is the per-token mask.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every data pointer is a DEVICE pointer (cudaMalloc'd or equivalent) owned
 *    by the caller. The library allocates nothing and keeps no state between
 *    calls besides cached kernel attributes and the driver entry point used
 *    to encode TMA descriptors.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream). Every call
 *    only enqueues work; it never synchronizes.
 *  - Layouts are row-major with the innermost dimension contiguous:
 *      X   bf16  [M, ldx]     (K used)            activations
 *      Xq  FP8:  uint8 [M, K] E4M3 codes;  NVFP4: uint8 [M, K/2] packed E2M1
 *          (element 2i in the low nibble of byte i)
 *      x_scale        fp32 [M]                     FP8 per-token scale
 *      x_block_scale  uint8 [M, K/16] E4M3         NVFP4 per-16-block scale
 *      x_global_scale fp32 scalar (device)         NVFP4 encode multiplier g_x
 *      Wq  FP8: uint8 [N, K];  NVFP4: uint8 [N, K/2]
 *      w_scale        fp32 [N]                     FP8 per-output-channel scale
 *      w_block_scale  uint8 [N, K/16];  w_global_scale fp32 scalar (device)
 *      A   bf16 [L, r, K]   (h = x A_l^T)
 *      B   bf16 [L, N, r]   (delta = h B_l^T)
 *      idx int32 [M]   adapter slot of each token; idx < 0 = no adapter
 *      mask uint8 [M]  0 = adapter skipped for this token; NULL = all ones
 *      S   fp32 [M, r]  shrink output (workspace)
 *      Y   bf16 [M, ldy] (N used)
 *  - Constraints (checked on the host before any launch; violation returns
 *    EPILORA_ERR_INVALID_ARG and enqueues nothing): M >= 0 (M == 0 is a
 *    no-op), K % 32 == 0 and K >= 32, N % 16 == 0 and N >= 16,
 *    r in {16, 32, 64, 128}, L >= 1, ldx >= K and ldx % 8 == 0,
 *    for NVFP4 GEMMs K % 256 == 0 (the block-scale rows must be 16-byte
 *    multiples for the tensor-memory-accelerator copies),
 *    ldy >= N and ldy % 8 == 0, every data pointer 16-byte aligned, the
 *    NVFP4 global scales non-NULL.
 *  - Device-detected conditions are written to the optional `status_dev`
 *    (int32 on the device, caller-owned; the first error wins through an
 *    atomic compare-and-swap of 0): an adapter index idx >= L makes that
 *    token "no adapter" and records EPILORA_ERR_INVALID_ARG; a non-positive
 *    or non-finite NVFP4 global scale records EPILORA_ERR_INVALID_ARG; a
 *    bounded wait inside a kernel that ran out records EPILORA_ERR_TIMEOUT
 *    (the kernel then releases its resources and returns; its outputs are
 *    undefined). Kernels never trap.
 *  - Results are deterministic: every reduction is summed in a fixed order
 *    (no floating-point atomics), so the same inputs at the same M give
 *    bitwise-identical outputs.
 *  - Errors from the CUDA runtime at launch are returned as EPILORA_ERR_CUDA.
 */
#ifndef EPILORA_H_
#define EPILORA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define EPILORA_API __attribute__((visibility("default")))
#else
#define EPILORA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  EPILORA_OK = 0,
  EPILORA_ERR_INVALID_ARG = -1,
  EPILORA_ERR_UNSUPPORTED = -2,
  EPILORA_ERR_CUDA = -3,
  EPILORA_ERR_TIMEOUT = -4,
  EPILORA_ERR_WORKSPACE = -5
} epilora_status;

typedef enum { EPILORA_FMT_FP8_E4M3 = 0, EPILORA_FMT_NVFP4 = 1 } epilora_format;

/* Smallest per-token amax used by the FP8 quantizer: an all-zero token gets
 * scale 1e-12f / 448 and all-zero codes. */
#define EPILORA_FP8_AMAX_FLOOR 1e-12f

/* Version of this ABI (bumped on any signature change). */
EPILORA_API int epilora_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
EPILORA_API const char* epilora_status_string(int status);

/*
 * Per-token activation quantizer (S1 / S1').
 * Defined by: EpiLoRA page, §Design › Multi-adapter kernels › K1 and K2
 * (activations are quantized one time per layer, with one scale per token,
 * for the low-precision base GEMM), and its Introduction / Related work for
 * the block-scaled 4-bit NVFP4 format.
 *
 * FP8:   s_t = fl32(max(amax_t, EPILORA_FP8_AMAX_FLOOR) / 448)  (IEEE division)
 *        Xq[t,k] = E4M3_rn_satfinite(fl32(X[t,k] / s_t));  x_scale[t] = s_t
 *        (x_block_scale, x_global_scale ignored; may be NULL)
 * NVFP4: per 16-element block b of token t, with g = *x_global_scale:
 *        sb = E4M3_rn_satfinite(fl32(fl32(amax_b / 6) * g));
 *        sb == 0 -> the block's codes are 0, else
 *        code = E2M1_rn_satfinite(fl32(X * fl32(g / sb)));
 *        x_block_scale[t,b] = sb (E4M3 byte)          (x_scale ignored)
 * Applied to a weight matrix (M := N rows) this also produces the FP8
 * per-output-channel weight scales and the NVFP4 weight codes, and applied to
 * the rows of adapter tables the stored FP8 adapters of
 * epilora_layer_forward_fp8_adapters (FP8 takes any K % 16 == 0, so rank-16
 * rows too). Codes and scales are bit-exact functions of the inputs.
 */
EPILORA_API int epilora_quant_act(int fmt, const void* X, int M, int K, int ldx,
                      void* Xq, float* x_scale, uint8_t* x_block_scale,
                      const float* x_global_scale, int* status_dev, void* stream);

/*
 * NVFP4 encode multiplier of a whole bf16 tensor of n elements:
 *   *g_out = fl32(448 * 6 / max(amax, EPILORA_FP8_AMAX_FLOOR)).
 * A load-time (weights) or calibration (activations) helper; the EpiLoRA
 * page only says NVFP4 has an fp32 global scale. g_out is a device float.
 */
EPILORA_API int epilora_nvfp4_global_scale(const void* T, size_t n, float* g_out, void* stream);

/*
 * Multi-adapter shrink (down-projection) (S2).
 * Defined by: EpiLoRA page, §Background and motivation › The cost of the
 * separate adapter path (h = x A^T) and §Design › Multi-adapter kernels ›
 * K1 and K2 (h from the bf16 activations); mask from the PreFT page.
 *   S[t, j] = sum_k X[t,k] * A[idx_t, j, k]   (fp32 accumulate, fixed order)
 * for tokens with idx_t in [0, L) and (mask == NULL or mask[t] != 0);
 * S[t, :] = 0 for every other token. Launched as an ordinary kernel (it
 * waits for X); it allows a dependent kernel to launch at once.
 */
EPILORA_API int epilora_lora_shrink(const void* X, int M, int K, int ldx,
                        const void* A, int L, int r,
                        const int32_t* idx, const uint8_t* mask,
                        float* S, int* status_dev, void* stream);

/*
 * Low-precision base GEMM with the multi-adapter LoRA epilogue (S3 + S5, S4).
 * Defined by: EpiLoRA page, §Design › Multi-adapter kernels › K1 and K2
 * (the epilogue applies the scales and adds h_l B_l^T for the rows of each
 * adapter) and › The decode path (launched as the shrink's dependent; waits
 * for h only before its epilogue).
 *   FP8:   Y[t,n] = bf16( (sum_k Xq[t,k] Wq[n,k]) * x_scale[t] * w_scale[n] + d[t,n] )
 *   NVFP4: Y[t,n] = bf16( (sum_k (Xq*sbx)[t,k] (Wq*sbw)[n,k]) / (g_x * g_w) + d[t,n] )
 *   d[t,n] = sum_j S[t,j] * B[idx_t, n, j] for active tokens (as in the
 *            shrink), else 0; with S == NULL there is no adapter term.
 * pdl_dependent = 1 launches the kernel with programmatic stream
 * serialization: it may start while the previous kernel on the stream (the
 * shrink) is still running, streams W and Xq at once, and executes the
 * grid-dependency wait before it reads x_scale, idx, mask or S.
 * pdl_dependent = 0 is an ordinary launch.
 * With pdl_dependent = 1, Xq and x_block_scale must already be complete when
 * the previous kernel on the stream started (e.g. written by
 * epilora_quant_act before the shrink); x_scale, S, idx and mask may be
 * written by that kernel.
 */
EPILORA_API int epilora_gemm_lora_epilogue(int fmt, int M, int N, int K,
                               const void* Xq, const float* x_scale,
                               const uint8_t* x_block_scale, const float* x_global_scale,
                               const void* Wq, const float* w_scale,
                               const uint8_t* w_block_scale, const float* w_global_scale,
                               const float* S, const void* B, int L, int r,
                               const int32_t* idx, const uint8_t* mask,
                               void* Y, int ldy, int pdl_dependent,
                               int* status_dev, void* stream);

/*
 * Bytes of device workspace epilora_layer_forward needs for (fmt, M, K, r):
 * a head of EPILORA_WORKSPACE_SYNC_BYTES (2.25 MiB: the single-kernel decode
 * path's launch counter and the regions where its thread blocks exchange
 * partial results, see epilora_layer_forward_kernels), then the quantized
 * activations, their scales, S (r = 0: no adapters; S is held as up to
 * ceil(K / 1024) partial sums over K slices, capped at 8) and, for more than
 * 32 tokens with adapters, a row-to-token map; each region 256-byte aligned.
 * Returns 0 for M == 0 or invalid arguments.
 */
#define EPILORA_WORKSPACE_SYNC_BYTES 2360576
EPILORA_API size_t epilora_workspace_bytes(int fmt, int M, int K, int r);

/*
 * Bytes of device workspace with which epilora_layer_forward (and _slices,
 * _noalloc) computes the adapter term of a batch of more than 32 tokens in a
 * pass of its own (the adapter kernels the EpiLoRA page runs after the base
 * GEMM above the decode batch sizes, §Design › Timed dispatch):
 * epilora_workspace_bytes(fmt, M, K, r) plus, for M > 32 and r >= 32, an
 * fp32 buffer of M x N (256-byte rounded) placed right after the regions
 * listed there. A call with more than 32 tokens and bf16 adapters of rank 32
 * or more (per slice) whose workspace_bytes reaches this size enqueues three
 * kernels instead of two: the shrink grid, the expand pass (S . B_l for
 * every sorted row with an adapter, 128 output columns per tile, each tile
 * inside one slice) as its programmatic dependent, and the GEMM as the
 * expand pass's programmatic dependent, whose epilogue adds the fp32 term to
 * the base value before the one rounding to bf16 (the term: bf16 tensor-core
 * MMAs of the B rows with S split exactly into three bf16 parts, fp32
 * accumulation). Otherwise (rank 16, or a smaller workspace) the GEMM's
 * epilogue computes the term itself; the two agree within the arithmetic
 * bound of the method. Other shapes: the same as epilora_workspace_bytes.
 * Returns 0 for M == 0 or invalid arguments.
 */
EPILORA_API size_t epilora_layer_workspace_bytes(int fmt, int M, int N, int K, int r);

/*
 * Number of kernels epilora_layer_forward (and _slices, _fp8_adapters,
 * _noalloc) enqueues for (fmt, M, K, r), r as for epilora_workspace_bytes
 * (rank times slices, 0 without adapters), under the current decode-path
 * policy (epilora_set_decode_path): 1 when the single-kernel decode path takes
 * the call, 2 otherwise (the shrink grid with its quantizer blocks, then the
 * GEMM as its programmatic dependent), for a workspace of
 * epilora_workspace_bytes; a workspace of epilora_layer_workspace_bytes adds
 * the expand pass (3) where that size exceeds epilora_workspace_bytes. The single kernel can take a few
 * tokens: M <= 8, FP8 with M * K <= 16384 (one token up to K = 16384, four at
 * K = 4096), NVFP4 with the bf16 rows within 40 KB (one token up to
 * K = 16384, two at K = 8192), as long as the shared memory of the call
 * leaves room for two weight stages (large M * r excludes it); the automatic
 * policy gives it the FP8 calls only. Returns 0 for invalid arguments.
 */
EPILORA_API int epilora_layer_forward_kernels(int fmt, int M, int K, int r);

/*
 * Decode-path policy for all later calls in the process (calls already
 * enqueued are not affected): which path epilora_layer_forward (and _slices,
 * _fp8_adapters, _noalloc) takes for calls the single kernel can run.
 *   EPILORA_DECODE_PATH_AUTO (the default): the single kernel for FP8 bases,
 *     the shrink grid and the GEMM for NVFP4 bases (on GB300 each is the
 *     faster of the two for its format at one token on the 8B layer);
 *   EPILORA_DECODE_PATH_SINGLE: the single kernel wherever it can run;
 *   EPILORA_DECODE_PATH_TWO: the shrink grid and the GEMM always.
 * Results agree between the paths within the arithmetic bound of the
 * method (the adapter term and the split-K sums are added in a different
 * order). Returns the previous policy, or EPILORA_ERR_INVALID_ARG (policy
 * unchanged) for another value.
 */
#define EPILORA_DECODE_PATH_AUTO 0
#define EPILORA_DECODE_PATH_SINGLE 1
#define EPILORA_DECODE_PATH_TWO 2
EPILORA_API int epilora_set_decode_path(int policy);

/*
 * Fused one-call layer (the decode path of the EpiLoRA page, §Design ›
 * Multi-adapter kernels › The decode path).
 *
 * A few tokens (epilora_layer_forward_kernels == 1) run as ONE persistent
 * kernel, a programmatic dependent of the previous kernel on the stream: it
 * streams Wq (and w_block_scale) at once, waits for that kernel, then every
 * thread block quantizes the activations (the arithmetic of
 * epilora_quant_act) over the K range of its own weight units, takes a fixed
 * share of the shrink work items (token, 4 ranks, K slice: the arithmetic of
 * epilora_lora_shrink split into partial sums), and finishes its share of
 * the output; the weight stream is split evenly over the SMs, a weight tile
 * split between thread blocks being summed in a fixed order. It lets the
 * next kernel on the stream launch as soon as all its thread blocks run.
 * Otherwise it enqueues two kernels,
 *   1. the shrink grid (the arithmetic of epilora_lora_shrink, split over K
 *      slices into partial sums; for more than 32 tokens, blocks of 16
 *      consecutive tokens carrying at most two adapters on the tensor
 *      cores) plus quantizer CTAs (the arithmetic of epilora_quant_act; for
 *      more than 32 tokens with adapters the rows of Xq are written in
 *      adapter-sorted order), launched as a programmatic dependent of the
 *      previous kernel on the stream: it lets the GEMM launch when its CTAs
 *      start (decode batches, or a grid that fits the GPU) or as they
 *      finish, and waits for that kernel's completion before reading
 *      anything, and
 *   2. the GEMM of epilora_gemm_lora_epilogue as its programmatic dependent:
 *      it starts streaming Wq (and w_block_scale) as soon as it is resident,
 *      and reads everything else only after the shrink grid has completed;
 * using `workspace` (>= epilora_workspace_bytes, 256-byte aligned) for the
 * head, Xq, scales, S and the row map; with more than 32 tokens, adapters and
 * a workspace of epilora_layer_workspace_bytes, the expand pass runs between
 * the two (see there). The head (the first
 * EPILORA_WORKSPACE_SYNC_BYTES) must be zero before the first call that uses
 * the workspace: zero-fill a workspace once after allocating it. Calls keep
 * the head valid for the next call (each adds 256 to a 64-bit launch
 * counter at bytes [16, 24) of the head, whose value at the start of a call
 * gives the tag of every value its thread blocks exchange, so older values
 * are never taken for new ones); nothing else needs an initial value. Y is the
 * same whatever the row order. Calls that share a workspace must be ordered
 * on one stream.
 * Because the GEMM may start while the kernel that precedes this call on the
 * stream is still running, that kernel must not write Wq or w_block_scale
 * (every other input, X included, may be its output).
 * A == NULL or B == NULL computes the base layer only. Graph-capturable: it
 * makes no allocation and no synchronizing call.
 */
EPILORA_API int epilora_layer_forward(int fmt, int M, int N, int K,
                          const void* X, int ldx,
                          const void* Wq, const float* w_scale,
                          const uint8_t* w_block_scale, const float* w_global_scale,
                          const float* x_global_scale,
                          const void* A, const void* B, int L, int r,
                          const int32_t* idx, const uint8_t* mask,
                          void* Y, int ldy,
                          void* workspace, size_t workspace_bytes,
                          int* status_dev, void* stream);

/*
 * Multi-slice projection (the EpiLoRA page, §Design › Multi-adapter kernels:
 * fused projections such as qkv or gate_up carry one adapter per slice):
 * epilora_layer_forward where output columns [slice_end[s-1], slice_end[s])
 * (slice_end[-1] = 0) take slice s's own rank-r adapter pair. A is bf16
 * [L, n_slices * r, K] (slice s's A rows at [s*r, (s+1)*r)), B stays
 * [L, N, r] (row n belongs to its column's slice). n_slices in 1..4;
 * slice_end (host memory, read during the call) ascending, every end but the
 * last a multiple of 128, the last == N. The workspace must hold
 * epilora_workspace_bytes(fmt, M, K, n_slices * r) bytes (with
 * epilora_layer_workspace_bytes(fmt, M, N, K, n_slices * r), batches of more
 * than 32 tokens take the expand pass). idx / mask select
 * one adapter slot per token for all slices. Other arguments and errors as
 * epilora_layer_forward (A and B are required).
 */
EPILORA_API int epilora_layer_forward_slices(int fmt, int M, int N, int K,
                          const void* X, int ldx,
                          const void* Wq, const float* w_scale,
                          const uint8_t* w_block_scale, const float* w_global_scale,
                          const float* x_global_scale,
                          const void* A, const void* B, int L, int r,
                          int n_slices, const int* slice_end,
                          const int32_t* idx, const uint8_t* mask,
                          void* Y, int ldy,
                          void* workspace, size_t workspace_bytes,
                          int* status_dev, void* stream);

/*
 * Stored FP8 adapters (EpiLoRA page, §Design › Multi-adapter kernels › K1
 * and K2: adapters may be kept in FP8 and are dequantized in registers):
 * epilora_layer_forward with the adapter tables as E4M3 codes and one fp32
 * scale per row,
 *   Aq uint8 [L, r, K], a_scale fp32 [L, r]   (rank j of adapter l over K)
 *   Bq uint8 [L, N, r], b_scale fp32 [L, N]   (output n of adapter l over r)
 *   S[t, j] = a_scale[l, j] * sum_k X[t, k] * E4M3(Aq[l, j, k])   (l = idx_t)
 *   d[t, n] = b_scale[l, n] * sum_j S[t, j] * E4M3(Bq[l, n, j])
 * (the codes and scales of each row as epilora_quant_act gives them for the
 * row). About half the adapter bytes of bf16 tables; the page reports that
 * part of its accuracy checks with stored adapters failed, so this is an
 * option for the caller, not a default. Decode batches only: M <= 32, else
 * EPILORA_ERR_UNSUPPORTED. Workspace as epilora_layer_forward (r as given);
 * other arguments, results and errors as there (all four adapter pointers
 * required).
 */
EPILORA_API int epilora_layer_forward_fp8_adapters(int fmt, int M, int N, int K,
                          const void* X, int ldx,
                          const void* Wq, const float* w_scale,
                          const uint8_t* w_block_scale, const float* w_global_scale,
                          const float* x_global_scale,
                          const uint8_t* Aq, const float* a_scale,
                          const uint8_t* Bq, const float* b_scale, int L, int r,
                          const int32_t* idx, const uint8_t* mask,
                          void* Y, int ldy,
                          void* workspace, size_t workspace_bytes,
                          int* status_dev, void* stream);

/*
 * Test hook of the single-kernel decode path: with on != 0, later calls that
 * take that path (in this process) have their shrink work items publish
 * nothing, so every finishing thread block that needs S waits until its
 * bounded wait runs out (1 s), records EPILORA_ERR_TIMEOUT in the status
 * word and returns in order (Y is then unspecified). on = 0 restores normal
 * operation. Not for production use; returns EPILORA_OK.
 */
EPILORA_API int epilora_test_drop_shrink_results(int on);

/*
 * epilora_layer_forward without a caller workspace. The EpiLoRA page has no
 * counterpart of this entry point: it serves callers that cannot hand the
 * library device memory, such as a plain C host with no device allocator of
 * its own, or code at a point where entering an allocator is not allowed (an
 * allocator's own hook, a section that must not call cudaMalloc).
 *
 * It allocates nothing. Its scratch is a fixed array of
 * EPILORA_NOALLOC_SCRATCH_BYTES bytes of static device storage inside the
 * library, one per device. The first call on a device (the device current
 * at the call) looks up that array's address with cudaGetSymbolAddress; make
 * that first call before any stream capture. Arguments, layout, results and
 * status codes are those of epilora_layer_forward without the workspace.
 *
 * Returns EPILORA_ERR_WORKSPACE, having enqueued nothing, when
 * epilora_workspace_bytes(fmt, M, K, A && B ? r : 0) exceeds
 * EPILORA_NOALLOC_SCRATCH_BYTES (8 MiB); the test is exactly that size query,
 * whose S term grows with the number of K slices of the shrink (e.g. FP8,
 * r = 64: M up to 1175 at K = 4096); EPILORA_ERR_CUDA if the address lookup
 * fails.
 * Otherwise it enqueues what epilora_layer_forward enqueues given a workspace
 * of the whole scratch (the scratch starts zeroed when the library is
 * loaded, which is what epilora_layer_forward requires of a workspace's
 * head): batches of more than 32 tokens with rank >= 32 take the expand pass
 * whenever epilora_layer_workspace_bytes fits the scratch.
 *
 * All calls on one device share the one scratch array: calls that overlap in
 * time (on different streams, or from host threads that do not order their
 * streams) race on it and produce wrong results. Order them on one stream.
 */
#define EPILORA_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
EPILORA_API int epilora_layer_forward_noalloc(int fmt, int M, int N, int K,
                          const void* X, int ldx,
                          const void* Wq, const float* w_scale,
                          const uint8_t* w_block_scale, const float* w_global_scale,
                          const float* x_global_scale,
                          const void* A, const void* B, int L, int r,
                          const int32_t* idx, const uint8_t* mask,
                          void* Y, int ldy,
                          int* status_dev, void* stream);

/* ------------------------------------------------------------------------
 * Attention of a decoder layer between its qkv and o projections: a paged
 * key/value cache, the kernel that appends to it, and the attention that
 * reads it; and the attention of whole packed prompts without a cache.
 *
 * Common to the three calls: `heads` query heads share `kv_heads` key/value
 * heads in groups of G = heads / kv_heads (query head h reads key/value head
 * h / G). Activations are bf16; Q, K, V and O are given by a pointer, a
 * token stride and a head stride in elements (the head_dim elements of a
 * head are contiguous; strides are multiples of 8, pointers 16-byte
 * aligned), so the slices of a fused qkv projection's output are used as
 * they are. No stride may make two elements of a written tensor coincide.
 * ------------------------------------------------------------------------ */
typedef enum { EPILORA_KV_BF16 = 0, EPILORA_KV_E4M3 = 1 } epilora_kv_format;

/*
 * A paged cache of one layer (this struct is host memory, read during the
 * call; k, v and the scales are device memory). Entry (page p, head g, token
 * row i of the page, element d) is at
 *   k[p * k_page_stride + g * k_head_stride + i * k_token_stride + d]
 * (strides in elements; the byte strides are multiples of 16, k and v
 * 16-byte aligned), v alike: pages of heads ("[page][head][token][d]") and
 * pages of tokens ("[page][token][head][d]") are both one choice of strides.
 * page_size is 16, 32, 64, 128 or 256 tokens, head_dim 64 or 128.
 * EPILORA_KV_E4M3: codes of one byte, the value is code * k_scale[g] (fp32
 * per head, device; required then, ignored for bf16).
 */
typedef struct {
  int kv_fmt;
  int kv_heads;
  int head_dim;
  int page_size;
  int num_pages;
  int reserved; /* 0 */
  void* k;
  void* v;
  int64_t k_page_stride, k_head_stride, k_token_stride;
  int64_t v_page_stride, v_head_stride, v_token_stride;
  const float* k_scale; /* [kv_heads] */
  const float* v_scale; /* [kv_heads] */
} epilora_kv_cache;

/*
 * The sequences of one step (host struct, device arrays). Sequence b owns
 * the packed new tokens q_start[b] .. q_start[b+1] - 1 (possibly none) and
 * holds kv_len[b] tokens once they are appended: its new token i stands at
 * position kv_len[b] - n_new + i. Position j is row j % page_size of page
 * page_table[b * table_stride + j / page_size]. q_start ascends from 0;
 * packed rows from q_start[n_seqs] up to n_tokens belong to no sequence
 * (padding of a captured graph). max_new is the caller's upper bound of the
 * new tokens of any sequence (n_tokens always is one): it selects kernels,
 * whose results differ by roundings within the bounds stated at the calls.
 * Device-detected, EPILORA_ERR_INVALID_ARG in the status word: q_start that
 * descends or leaves [0, n_tokens], more new tokens than max_new, kv_len
 * beyond table_pages * page_size, a page index that is read and is outside
 * [0, num_pages). No access is made out of bounds then; the outputs of the
 * sequences concerned are unspecified.
 */
typedef struct {
  int n_seqs;
  int n_tokens;
  int max_new;
  int table_pages;  /* columns of page_table in use */
  int64_t table_stride;
  const int32_t* q_start;    /* [n_seqs + 1] */
  const int32_t* kv_len;     /* [n_seqs] */
  const int32_t* page_table; /* [n_seqs][table_stride] */
} epilora_kv_batch;

/*
 * Appends the new tokens' keys and values to the cache, rotating queries and
 * keys by their position on the way.
 * For a token at position p, each q and k head row x with c = cos_sin[p][i],
 * s = cos_sin[p][rot_dim / 2 + i], i in [0, rot_dim / 2), fp32 arithmetic
 * with one rounding per operation:
 *   y[a] = fl(fl(x[a] c) - fl(x[b] s)),  y[b] = fl(fl(x[b] c) + fl(x[a] s))
 *   (a, b) = (i, i + rot_dim / 2), or (2i, 2i + 1) with interleaved != 0;
 * elements from rot_dim on are copied. Qout takes bf16(y). The cache takes
 * bf16(y) of k and v itself, or E4M3_rn_satfinite(fl(y / k_scale[g])) and
 * E4M3_rn_satfinite(fl(v / v_scale[g])): bit-exact functions of the inputs.
 * cos_sin is fp32 [n_pos][rot_dim] (cosines, then sines), rot_dim a multiple
 * of 16 up to head_dim; cos_sin == NULL rotates nothing (Q, Qout may then be
 * NULL too). Qout may be Q itself (same strides); otherwise it must not
 * overlap Q, K or V.
 * A token of no sequence, at a negative position (more new tokens than
 * kv_len), or that fails a device check (the above, or a position >= n_pos)
 * appends nothing; its Qout rows are zero. The new tokens of a batch have to
 * go to different cache rows. n_tokens == 0 is a no-op. One kernel, a
 * programmatic dependent of the previous kernel on the stream (it waits for
 * that kernel before it reads anything).
 */
EPILORA_API int epilora_kv_append(const epilora_kv_cache* cache, const epilora_kv_batch* batch, int heads,
                      const void* Q, int64_t q_token_stride, int64_t q_head_stride,
                      const void* K, int64_t k_token_stride, int64_t k_head_stride,
                      const void* V, int64_t v_token_stride, int64_t v_head_stride,
                      const float* cos_sin, int n_pos, int rot_dim, int interleaved,
                      void* Qout, int64_t qo_token_stride, int64_t qo_head_stride,
                      int* status_dev, void* stream);

/*
 * Bytes of device workspace epilora_paged_attention and
 * epilora_prompt_attention need (the partial results of sequences that
 * several thread blocks share). It depends on the device's number of SMs and
 * on head_dim only, so one workspace serves every layer and step of a model
 * (head_dim 128 needs more than 64, and the larger serves both).
 * Zero-fill its first epilora_attention_workspace_zero_bytes() bytes, or all
 * of it, once after allocating it; calls leave it ready for the next one
 * (after a call that recorded EPILORA_ERR_TIMEOUT, zero it again). A fill that
 * a stream capture records is run by the graph alone: fill before the capture.
 * Calls that share a workspace must be ordered on one stream. Returns 0 for a
 * head_dim other than 64 or 128.
 */
EPILORA_API size_t epilora_attention_workspace_bytes(int head_dim);

/* Bytes at the head of that workspace that have to be zero before a call
 * (counters; what follows is written before it is read). */
EPILORA_API size_t epilora_attention_workspace_zero_bytes(void);

/*
 * Attention of the new tokens over the paged cache (their own keys and
 * values appended before): for token t of sequence b at position p,
 *   x_j = scale * q[t,h] . K[b, j, h / G],  j in [0, p]
 *   O[t,h] = bf16( sum_j exp(x_j - m) V[b, j, h / G] / sum_j exp(x_j - m) )
 *   lse[t,h] = ln sum_j exp(x_j)   (fp32 [n_tokens][heads], optional)
 * with scores, statistics and sums in fp32 (the weights exp(x_j - m) are
 * rounded to the tensor cores' 16-bit operand type: bf16, or fp16 for an
 * E4M3 cache; an E4M3 cache's queries are scaled by a power of two per row
 * into fp16, and its weights are taken times 2^7: those below 2^-21 of the
 * largest are off by up to 2^-32 of it). A row that sees nothing (negative
 * position, no sequence) is zero, its lse -infinity. What a masked position,
 * a page's unused rows or an unused page hold never reaches a result, NaN and
 * infinities included. scale is finite. O must not overlap any input.
 * Kernels: one for the sequences whose new tokens times G are at most 16
 * rows; where max_new * G exceeds that, a second one for the others, which
 * starts as the first one's blocks end, or alone where n_tokens is
 * n_seqs * max_new. Programmatic dependents of the
 * previous kernel on the stream, like epilora_kv_append. The results of the
 * same call (max_new included) are the same from run to run.
 * n_tokens * heads has to stay below 2^30 (EPILORA_ERR_UNSUPPORTED);
 * n_tokens == 0 is a no-op.
 */
EPILORA_API int epilora_paged_attention(const epilora_kv_cache* cache, const epilora_kv_batch* batch, int heads,
                      const void* Q, int64_t q_token_stride, int64_t q_head_stride, float scale,
                      void* O, int64_t o_token_stride, int64_t o_head_stride, float* lse,
                      void* workspace, size_t workspace_bytes, int* status_dev, void* stream);

/*
 * Causal attention of whole packed prompts, keys and values straight from
 * the projection: prompt b is the packed rows q_start[b] .. q_start[b+1] - 1
 * of Q, K and V; row i of a prompt attends to its rows 0 .. i. Results and
 * conventions as epilora_paged_attention (q_start as in epilora_kv_batch).
 * One kernel.
 */
EPILORA_API int epilora_prompt_attention(int n_seqs, int n_tokens, const int32_t* q_start,
                      int heads, int kv_heads, int head_dim,
                      const void* Q, int64_t q_token_stride, int64_t q_head_stride,
                      const void* K, int64_t k_token_stride, int64_t k_head_stride,
                      const void* V, int64_t v_token_stride, int64_t v_head_stride, float scale,
                      void* O, int64_t o_token_stride, int64_t o_head_stride, float* lse,
                      void* workspace, size_t workspace_bytes, int* status_dev, void* stream);

/* ------------------------------------------------------------------------
 * Projections and mixtures of experts in 8-bit blocks: E4M3 codes with one
 * fp32 scale per 128 consecutive elements of an activation row, and one per
 * 128 x 128 block of a weight (the last block of a row or column may be
 * shorter). nb(n) below is ceil(n / 128).
 *   activation codes  uint8 [M][K]          scale fp32 [nb(K)][x_scale_ld], scale[b][m]
 *   weight codes      uint8 [N][K]          scale fp32 [nb(N)][nb(K)]
 * Widths (K, and hidden and inner of a mixture) are multiples of 16; M and N
 * are any. No size exceeds EPILORA_BLOCK_MAX_SIZE, nor does the sum of the rows
 * of all experts' weights (EPILORA_ERR_UNSUPPORTED). Code arrays and bf16 inputs are 16-byte aligned, bf16 rows have
 * strides in multiples of 8 elements. All calls are forward only. Their
 * kernels are programmatic dependents of the previous kernel on the stream
 * and wait for it before they read anything it may have written. A wait
 * inside a product that runs out (1 s; no call does that) records
 * EPILORA_ERR_TIMEOUT in the status word; the results that it left unfinished
 * are NaN, and so is what is computed from them.
 * ------------------------------------------------------------------------ */

#define EPILORA_BLOCK_MAX_SIZE 0x7fff0000

/*
 * Codes and scales of bf16 rows X [M][ldx], per block b of 128 elements:
 *   s = fl32(max(amax_b, EPILORA_FP8_AMAX_FLOOR) / 448),
 *   code = E4M3_rn_satfinite(fl32(x / s)),
 * bit-exact functions of the inputs. A NaN element gets the code of NaN and
 * does not count in amax; an infinity makes the block's scale infinite and
 * its own code NaN. One kernel. M == 0 is a no-op.
 */
EPILORA_API int epilora_block_quant(const void* X, int M, int K, int64_t ldx, uint8_t* Xq, float* x_scale,
                      int64_t x_scale_ld, void* stream);

/* The same for a weight W [N][ldw], one scale per 128 x 128 block (load time). */
EPILORA_API int epilora_block_quant_weight(const void* W, int N, int K, int64_t ldw, uint8_t* Wq, float* w_scale,
                      void* stream);

/*
 * Y[m][n] = bf16( sum_b x_scale[b][m] w_scale[n / 128][b] sum_{k in b} Xq[m][k] Wq[n][k] )
 * with fp32 sums: the products of a block on the tensor cores, then the
 * blocks in order (up to 32 rows with long K: the blocks of up to eight parts
 * of K in order, then the parts). A NaN in a row of Xq or Wq reaches that
 * row's or column's results alone. Y is bf16 [M][ldy], ldy >= N, of any
 * alignment (rows of 32-byte aligned starts are written faster), and must not
 * overlap an input. One kernel. M == 0 is a no-op.
 */
EPILORA_API int epilora_block_matmul(int M, int N, int K, const uint8_t* Xq, const float* x_scale, int64_t x_scale_ld,
                      const uint8_t* Wq, const float* w_scale, void* Y, int64_t ldy, int* status_dev, void* stream);

/* epilora_block_quant of X into the workspace, then epilora_block_matmul:
 * two kernels, the second of which reads its first weights while the first
 * runs (and everything before that is done). The workspace (256-byte aligned) needs no initialization;
 * calls that share one must be ordered on one stream. */
EPILORA_API size_t epilora_block_linear_workspace_bytes(int M, int K);
EPILORA_API int epilora_block_linear(int M, int N, int K, const void* X, int64_t ldx, const uint8_t* Wq,
                      const float* w_scale, void* Y, int64_t ldy, void* workspace, size_t workspace_bytes,
                      int* status_dev, void* stream);

/*
 * Test hook of the products in 8-bit blocks: with on != 0, later calls (in
 * this process) expect more bytes than they copy for the last block of K of a
 * tile, so that the waits for it run out (some seconds a call). on = 0 restores
 * normal operation. Not for production use; returns EPILORA_OK.
 */
EPILORA_API int epilora_test_late_block_copies(int on);

#define EPILORA_MOE_MAX_EXPERTS 1024
#define EPILORA_MOE_MAX_TOP 32
typedef enum { EPILORA_LOGITS_F32 = 0, EPILORA_LOGITS_BF16 = 1 } epilora_logits_format;
typedef enum { EPILORA_SCORE_SOFTMAX = 0, EPILORA_SCORE_SIGMOID = 1 } epilora_scoring;

/*
 * Chooses `top` experts for each token from its logits (row t at
 * logits + t * ld, fp32 or bf16).
 *   score s_e = softmax over the experts, or sigmoid, of the logits
 *   choice c_e = s_e + bias[e]   (bias fp32 [experts] or NULL)
 *   groups > 1: expert e belongs to group e / (experts / groups); a group's
 *     value is the sum of its `group_best` (1 or 2) largest c, and only the
 *     `top_groups` groups of the largest values stay (ties: lowest index)
 *   ids[t][0 .. top): the experts of the largest c among those, descending.
 *     c is compared in 64 bits; where those are equal (scores that a bias or a
 *     1 swallows) the larger logit goes first, then the lowest index. With
 *     equal biases, or none, that is the order of the real numbers c
 *   weights[t][j] = scale * s of the j-th, divided by the sum of the chosen
 *     s first if renormalize, in fp32
 * A logit of -infinity or NaN, or a bias of -infinity or NaN, takes the
 * expert away for that token; +infinity counts as the largest finite number.
 * Slots for which no expert is left have id -1 and weight 0.
 * experts <= EPILORA_MOE_MAX_EXPERTS, a multiple of groups; groups <= 32;
 * top <= EPILORA_MOE_MAX_TOP and <= top_groups * experts / groups. One kernel.
 */
EPILORA_API int epilora_moe_route(int tokens, int experts, int top, const void* logits, int logits_fmt, int64_t ld,
                      const float* bias, int scoring, int groups, int top_groups, int group_best, int renormalize,
                      float scale, int32_t* ids, float* weights, void* stream);

/*
 * The gated MLPs of a mixture's experts. Slot j of token t (number
 * t * top + j) goes to expert e = ids[t][j]; a negative id is no expert, and
 * so is one >= experts, which also records EPILORA_ERR_INVALID_ARG in the
 * status word. A token may name an expert twice.
 *   Wup   codes [experts][2][inner][hidden], scale [experts][2][nb(inner)][nb(hidden)]  (gate, then up)
 *   Wdown codes [experts][hidden][inner],    scale [experts][nb(hidden)][nb(inner)]
 * up:   x is block-quantized; h = silu(x Wup[e][0]^T) * (x Wup[e][1]^T), silu(g) = g / (1 + exp(-g)), in fp32,
 *       silu within 2^-21 + |g| 2^-24 of its value (0 below g = -87.3, where it is less than 2^-119);
 *       Hq [tokens][top][inner] and h_scale [nb(inner)][tokens * top] are its
 *       block quantization; slots without an expert: zero codes, zero scales
 * down: Y[t] = bf16( sum_j weights[t][j] bf16(h[t][j] Wdown[e]^T) ), j ascending in fp32 over the slots that
 *       have an expert (each expert's output is rounded to bf16 once, as a model that adds them up would)
 * epilora_moe_experts_down_f32 and epilora_moe_experts_f32 keep each expert's output in fp32 and round Y alone; they
 * write and read 8 bytes instead of 4 per slot and column of Y on the way, in a larger workspace.
 * epilora_moe_experts is up, then down. X is bf16 [tokens][ldx], Y bf16
 * [tokens][ldy], 16-byte aligned, ldy a multiple of 8; outputs must not
 * overlap inputs. Kernels: up 3, down 4, both 5. Which kernels run depends on
 * the sizes alone, and a token's results on no other token. tokens == 0 is a
 * no-op.
 * Workspace: epilora_moe_workspace_bytes(what, ...) bytes for EPILORA_MOE_UP,
 * EPILORA_MOE_DOWN, or both or'ed together for epilora_moe_experts, with
 * EPILORA_MOE_F32_PARTS or'ed to the last two for the _f32 calls; 256-byte
 * aligned, no initialization; calls that share one must be ordered on one
 * stream. 0 for sizes that the calls refuse.
 */
typedef enum { EPILORA_MOE_UP = 1, EPILORA_MOE_DOWN = 2, EPILORA_MOE_F32_PARTS = 4 } epilora_moe_part;
EPILORA_API size_t epilora_moe_workspace_bytes(int what, int tokens, int top, int experts, int hidden, int inner);
EPILORA_API int epilora_moe_experts_up(int tokens, int top, int experts, int hidden, int inner,
                      const void* X, int64_t ldx, const int32_t* ids, const uint8_t* Wup, const float* wup_scale,
                      uint8_t* Hq, float* h_scale, void* workspace, size_t workspace_bytes, int* status_dev,
                      void* stream);
EPILORA_API int epilora_moe_experts_down(int tokens, int top, int experts, int hidden, int inner,
                      const uint8_t* Hq, const float* h_scale, const int32_t* ids, const float* weights,
                      const uint8_t* Wdown, const float* wdown_scale, void* Y, int64_t ldy,
                      void* workspace, size_t workspace_bytes, int* status_dev, void* stream);
EPILORA_API int epilora_moe_experts_down_f32(int tokens, int top, int experts, int hidden, int inner,
                      const uint8_t* Hq, const float* h_scale, const int32_t* ids, const float* weights,
                      const uint8_t* Wdown, const float* wdown_scale, void* Y, int64_t ldy,
                      void* workspace, size_t workspace_bytes, int* status_dev, void* stream);
EPILORA_API int epilora_moe_experts(int tokens, int top, int experts, int hidden, int inner,
                      const void* X, int64_t ldx, const int32_t* ids, const float* weights,
                      const uint8_t* Wup, const float* wup_scale, const uint8_t* Wdown, const float* wdown_scale,
                      void* Y, int64_t ldy, void* workspace, size_t workspace_bytes, int* status_dev, void* stream);
EPILORA_API int epilora_moe_experts_f32(int tokens, int top, int experts, int hidden, int inner,
                      const void* X, int64_t ldx, const int32_t* ids, const float* weights,
                      const uint8_t* Wup, const float* wup_scale, const uint8_t* Wdown, const float* wdown_scale,
                      void* Y, int64_t ldy, void* workspace, size_t workspace_bytes, int* status_dev, void* stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* EPILORA_H_ */
