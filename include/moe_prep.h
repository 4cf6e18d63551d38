/*
 * moe_prep.h -- C ABI of the GB300 (sm_103a) batched grouped-masked block-FP8
 * MoE expert forward.
 *
 * Three entry points make up the path:
 *
 *   moe_prepare_inputs   input staging: bf16 -> fp8 e4m3 with 1x128 UE8M0
 *                        scales, top-k repack (int64 ids, fp32 weights),
 *                        EPLB replica map, and optionally the dispatch into
 *                        the batched [experts, max_tokens, K] layout.
 *   moe_batched_experts  w13 gate_up GEMM masked by expert_num_tokens, fused
 *                        SiLU-and-mul + FP8 requant, w2 down GEMM.
 *   moe_topk_reduce      top-k weighted sum back to token order.
 *
 * Around them stand the other operators of an MoE block, for serving and for
 * training, in bf16, fp16 and fp32:
 *
 *   moe_route            router logits -> top-k ids and weights (and the
 *                        gradient of the logits).
 *   moe_sort_routes, moe_permute, moe_unpermute
 *                        rows sorted by expert and back with the routing
 *                        weights applied (and their gradients).
 *   moe_block_norm       the RMS norm after a block with its gate, residual
 *                        scale and residual sum, and the norm before the next
 *                        block, in one pass (and its gradient).
 *   moe_norm_quant       the norm before a block with its output in 8 bits, as
 *                        the experts take it.
 *   moe_lora_linear      a projection shared by all tokens plus each token's
 *                        own low-rank adapter.
 *   moe_gated_linear     gate and up projections with the activation and the
 *                        product in one kernel (and its gradients).
 *   moe_w4_linear        products of few rows with 4-bit weights and group
 *                        scales, of one matrix or of each row's expert.
 *
 * Conventions shared by every call
 *   - All tensor pointers are DEVICE pointers unless stated otherwise; every
 *     output buffer is allocated by the caller; the library never allocates
 *     device memory.
 *   - Strides are in ELEMENTS of the tensor's own dtype.
 *   - `stream` is a cudaStream_t passed as void*.  Work is enqueued
 *     asynchronously; nothing synchronises the host.
 *   - Host-checkable problems return a moe_status_t before anything is
 *     enqueued; moe_last_error() then holds a message (thread-local).
 *   - Problems only the device can see (an expert receiving more routes than
 *     it has rows, a routed id outside [0, num_experts), a GEMM wait that
 *     timed out) are OR-ed into *device_status (MOE_DEV_* bits) when the
 *     caller passes one.  Kernels never trap.
 */
#ifndef MOE_PREP_H
#define MOE_PREP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Changes with an existing signature, structure or result; entry points that are added keep it
 * and are found by their names. */
#define MOE_PREP_ABI_VERSION 3

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARGUMENT = 1, /* NULL where required, negative size, bad enum */
  MOE_ERR_SHAPE = 2,            /* a shape rule of the pages is broken */
  MOE_ERR_UNSUPPORTED = 3,      /* a combination this library does not implement */
  MOE_ERR_ALIGNMENT = 4,        /* pointer/stride alignment needed by vector or TMA access */
  MOE_ERR_WORKSPACE = 5,        /* workspace missing or smaller than the size query */
  MOE_ERR_CUDA = 6              /* a CUDA runtime call failed */
} moe_status_t;

/* Device status bits (OR-ed into *device_status). */
#define MOE_DEV_CAPACITY 1u   /* an expert got more than max_tokens_per_expert routes */
#define MOE_DEV_BAD_EXPERT 2u /* routed id >= num_experts / num_logical, or bad EPLB entry */
#define MOE_DEV_TIMEOUT 4u    /* a bounded pipeline wait inside a GEMM expired */
#define MOE_DEV_BAD_ADAPTER 8u /* an adapter id >= num_adapters (taken as no adapter) */

typedef enum moe_sf_mode {
  MOE_SF_NONE = 0,         /* no quantisation: x receives a bf16 copy of hidden */
  MOE_SF_UE8M0_PACKED = 1, /* x_sf int32 [T, ceil(G/4)]: group g is byte g%4 of word g/4 */
  MOE_SF_FP32 = 2          /* x_sf fp32 [T, G]: the group scale amax/448 itself */
} moe_sf_mode_t;

typedef enum moe_ids_dtype { MOE_IDS_INT32 = 0, MOE_IDS_INT64 = 1 } moe_ids_dtype_t;
typedef enum moe_weights_dtype { MOE_WEIGHTS_FP32 = 0, MOE_WEIGHTS_BF16 = 1 } moe_weights_dtype_t;
typedef enum moe_activation {
  MOE_ACT_SILU = 0,
  MOE_ACT_GELU_TANH = 1, /* 0.5 g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) */
  MOE_ACT_NONE = 2       /* moe_w4_linear: no gate */
} moe_activation_t;
typedef enum moe_shared_dtype { MOE_SHARED_BF16 = 0, MOE_SHARED_FP8 = 1 } moe_shared_dtype_t;
typedef enum moe_dtype { MOE_DTYPE_FP32 = 0, MOE_DTYPE_BF16 = 1, MOE_DTYPE_FP16 = 2 } moe_dtype_t;
typedef enum moe_w4_format {
  MOE_W4_INT4 = 0, /* q - zero point (8 without one), scales of the tensors' type */
  MOE_W4_E2M1 = 1  /* sign, two bits of exponent, one of mantissa; scales 2^(byte - 127) */
} moe_w4_format_t;
typedef enum moe_scoring {
  MOE_SCORE_SOFTMAX = 0,
  MOE_SCORE_SIGMOID = 1,
  /* OR-ed to SOFTMAX: moe_route's bias is added to the score, not to the logit (SIGMOID's always
   * is).  Without a bias, and to the gradient, it says nothing. */
  MOE_SCORE_BIAS_ON_SCORE = 4
} moe_scoring_t;
typedef enum moe_gate {
  MOE_GATE_NONE = 0,
  MOE_GATE_CHANNEL = 1, /* [K]: one factor per column */
  MOE_GATE_TOKEN = 2,   /* [T]: one factor per token */
  MOE_GATE_FULL = 3     /* [T, K] */
} moe_gate_t;

/* Stage mask of moe_batched_experts. */
#define MOE_STAGE_W13 1
#define MOE_STAGE_W2 2
#define MOE_STAGE_ALL 3

/* ------------------------------------------------------------------------ */
/* moe_prepare_inputs                                                        */
/*                                                                           */
/* Defined by prepare_megamoe_inputs, _quantize_fp8_groups, _pack_bytes,     */
/* _store_topk and _eplb_kernel_args on the page                             */
/* "vllm.model_executor.layers.fused_moe.prepare_megamoe", and, for the      */
/* optional dispatch, by the batched activation format of                    */
/* BatchedHummingGroupedExperts ("...fused_moe.experts.fused_humming_moe":   */
/* hidden_states [E, max_tokens, K] with expert_tokens_meta.expert_num_tokens).*/
/*                                                                           */
/* Per token t and 1x128 group g of hidden (G = K/128 groups):               */
/*   amax = max(max|x|, 1e-4); s = amax / 448 (fp32);                        */
/*   UE8M0: e = expfield(s) + (mantissa(s) != 0), clamped to [1, 254],       */
/*          qs = 2^(e-127);  FP32: qs = s;                                    */
/*   x[t, i] = e4m3_rn_satfinite(hidden[t, i] * (1 / qs)).                   */
/* Top-k: topk_idx_out = int64(topk_ids), topk_weights_out = fp32(weights);  */
/* padding tokens (is_padding[t] != 0) get id -1 and weight 0.               */
/* EPLB (when logical_to_physical != NULL) maps a routed logical id l to     */
/* logical_to_physical[l * map_stride + (t mod logical_replica_count[l])]    */
/* and, when *should_record != 0 and t < *num_unpadded_tokens, adds 1 to     */
/* expert_load[physical id].                                                 */
/* Dispatch (when x_b != NULL; UE8M0 or FP32 scales): routes are            */
/* placed in (token, k) order; route (t, j) with id e takes slot s, the      */
/* number of earlier routes to e, and x_b[e, s, :] = x[t, :],                */
/* sf_b[e, s, :] = x_sf[t, :], route_slot[t, j] = s (-1 when unrouted or     */
/* when s >= max_tokens_per_expert, which also sets MOE_DEV_CAPACITY),       */
/* expert_num_tokens[e] = min(#routes to e, max_tokens_per_expert).          */
/* Contiguous layout (when expert_offsets != NULL; the expert_offsets /     */
/* moe_permute layout of HummingGroupedExperts.apply on the experts page):  */
/* no per-expert capacity; the routes of expert e fill rows                 */
/* [expert_offsets[e], expert_offsets[e+1]) of x_b / sf_b in the same       */
/* (token, k) order, expert_offsets[e] = #routes to experts < e,            */
/* expert_offsets[E] = #routes, route_slot[t, j] = the row (not the slot)   */
/* and expert_num_tokens[e] the full count.  x_b / sf_b hold                */
/* E * max_tokens_per_expert rows, which must be >= T * k (else SHAPE).     */
/*                                                                           */
/* Shared-expert scale pages (when shared_x_sf != NULL; defined by the      */
/* shared_x_sf / shared_block_m arguments of prepare_megamoe_inputs and by   */
/* _shared_sf_row on the same page; requires MOE_SF_UE8M0_PACKED): the      */
/* exponent byte e of group g of token t is also written to                  */
/*   shared_x_sf[row(t) * shared_x_sf_stride0 + g * shared_x_sf_stride1],   */
/* one uint8 per (row, group) (reading: the page's UE8M0 scale element is    */
/* its exponent byte).  With B = shared_block_m, A = ceil(B/128)*128,        */
/* b = t / B and m = t % B:                                                  */
/*   row(t) = b*A + (m/128)*128 + (m%32)*4 + (m%128)/32,                     */
/* i.e. each 128-row page interleaves its four 32-token quarters row by row */
/* (the MN-major layout a tcgen05.cp of the scales expects).  Rows that no   */
/* token maps to are left untouched.  The buffer must hold at least         */
/* ceil(T/B)*A rows (shared_x_sf_rows), else SHAPE.                          */
/*                                                                           */
/* Errors: T == 0 -> MOE_OK, nothing enqueued.  K % 128 != 0 -> SHAPE.       */
/* x_sf given iff sf_mode != NONE, else INVALID_ARGUMENT.  top_k < 1 ->       */
/* SHAPE.  hidden / x rows must start on 16-byte boundaries (ALIGNMENT).     */
/* Dispatch needs workspace of moe_prepare_workspace_size() bytes (WORKSPACE)*/
/* and top_k <= 32 (UNSUPPORTED).                                            */
/* ------------------------------------------------------------------------ */
typedef struct moe_prepare_args {
  int64_t num_tokens;  /* T >= 0 */
  int64_t hidden_size; /* K, multiple of 128 */
  int64_t top_k;       /* k >= 1 */

  const void* hidden; /* bf16 [T, K], inner stride 1 */
  int64_t hidden_stride0;
  const void* topk_ids; /* int32 or int64 [T, k] */
  int32_t topk_ids_dtype;
  int64_t topk_ids_stride0, topk_ids_stride1;
  const void* topk_weights; /* fp32 or bf16 [T, k] */
  int32_t topk_weights_dtype;
  int64_t topk_weights_stride0, topk_weights_stride1;
  const uint8_t* is_padding; /* nullable; [T], nonzero = padding */
  int64_t is_padding_stride0;

  void* x; /* fp8 e4m3 [T, K] (bf16 when sf_mode == MOE_SF_NONE), inner stride 1 */
  int64_t x_stride0;
  void* x_sf; /* NULL iff sf_mode == MOE_SF_NONE */
  int32_t sf_mode;
  int64_t x_sf_stride0, x_sf_stride1;
  uint8_t* shared_x_sf;    /* nullable; UE8M0 exponent bytes [shared_x_sf_rows, K/128] */
  int64_t shared_x_sf_stride0, shared_x_sf_stride1;
  int64_t shared_x_sf_rows; /* rows of shared_x_sf */
  int64_t shared_block_m;   /* > 0 iff shared_x_sf != NULL */
  int64_t* topk_idx_out; /* int64 [T, k] */
  int64_t topk_idx_out_stride0, topk_idx_out_stride1;
  float* topk_weights_out; /* fp32 [T, k] */
  int64_t topk_weights_out_stride0, topk_weights_out_stride1;

  /* EPLB: all NULL / 0 leaves ids unmapped. */
  const int32_t* logical_to_physical; /* [num_logical, map_stride] */
  int64_t num_logical, map_stride;
  const int32_t* logical_replica_count; /* [num_logical], each >= 1 */
  int32_t* expert_load;                 /* nullable; [num_physical] */
  int64_t num_physical;
  const uint8_t* should_record;       /* nullable device scalar; NULL = never record */
  const int32_t* num_unpadded_tokens; /* nullable device scalar; NULL = T */

  /* Optional dispatch into the batched layout (x_b == NULL disables it). */
  int64_t num_experts;           /* E */
  int64_t max_tokens_per_expert; /* M_max */
  void* x_b;                     /* fp8 [E, M_max, K] */
  void* sf_b;                    /* int32 [E, M_max, ceil(G/4)] packed UE8M0, or fp32 [E, M_max, G] */
  int32_t* expert_num_tokens;    /* int32 [E] */
  int32_t* route_slot;           /* int32 [T, k], contiguous */
  int32_t* expert_offsets;       /* nullable int32 [E + 1]: contiguous layout */
  void* workspace;               /* moe_prepare_workspace_size() bytes */
  size_t workspace_bytes;

  uint32_t* device_status; /* nullable; MOE_DEV_* bits are OR-ed in */
} moe_prepare_args_t;

moe_status_t moe_prepare_inputs(const moe_prepare_args_t* args, void* stream);

/* Bytes of workspace the dispatch of moe_prepare_inputs needs. */
size_t moe_prepare_workspace_size(int64_t num_tokens, int64_t top_k, int64_t num_experts);

/* ------------------------------------------------------------------------ */
/* moe_prepare_nvfp4_inputs                                                  */
/*                                                                           */
/* Defined by prepare_megamoe_nvfp4_inputs (kNvfp4DynamicToken) on the page  */
/* "vllm.model_executor.layers.fused_moe.prepare_megamoe": each token is     */
/* scaled by its own fp32 x_scales (row amax / 2688) and quantised to E2M1   */
/* with one E4M3 scale per 16 values.  The kernel body is not on the page;  */
/* this library computes, in fp32 with IEEE roundings, per token t:          */
/*   xs = amax / 2688;  v_i = x_i * (1 / xs);                                */
/*   per 16 values: s = e4m3_rn_satfinite(max|v_i| / 6),                     */
/*                  q_i = e2m1_rn_satfinite(v_i * (1 / dec(s)));             */
/* amax == 0 gives xs = 0 and zero codes and scales; a block whose scale    */
/* rounds to 0 gets zero codes.  x: uint8 [T, K/2], value 2i in the low     */
/* nibble of byte i; x_sf: int32 [T, K/64], block b's E4M3 byte at byte     */
/* b % 4 of word b / 4; x_scales: fp32 [T].                                  */
/* Routing outputs (topk_idx_out, topk_weights_out, EPLB map and load) are  */
/* exactly those of moe_prepare_inputs.  Shared-expert input (the page's    */
/* shared_x, nullable), by shared_x_dtype:                                   */
/*   MOE_SHARED_BF16: bf16 [T, K], a copy of the hidden rows;                */
/*   MOE_SHARED_FP8 (MXFP8 with shared_x_sf): fp8 e4m3 [T, K], the hidden    */
/*     rows quantised exactly as moe_prepare_inputs quantises x (1x128        */
/*     groups, UE8M0 scales), and each group's exponent byte written to      */
/*     shared_x_sf at row(t) of the shared-expert pages of shared_block_m     */
/*     (the same layout and row rule as moe_prepare_inputs' shared_x_sf).    */
/* shared_x_sf and shared_block_m are given exactly for an fp8 shared_x      */
/* (else INVALID_ARGUMENT, as the page raises); shared_x_sf must hold         */
/* ceil(T/B)*A rows (SHAPE).                                                 */
/* l2_alpha[e] = w2_global_scale[e] * l2_activation_scale for e <            */
/* num_local_experts, written even when T == 0 (both NULL or both given).    */
/* Errors: K % 128 != 0 -> SHAPE; rows of hidden, x, shared_x not 16-byte    */
/* aligned -> ALIGNMENT; w2_global_scale without l2_alpha -> INVALID.        */
/* ------------------------------------------------------------------------ */
typedef struct moe_nvfp4_args {
  int64_t num_tokens, hidden_size, top_k;
  const void* hidden; /* bf16 [T, K] */
  int64_t hidden_stride0;
  const void* topk_ids;
  int32_t topk_ids_dtype;
  int64_t topk_ids_stride0, topk_ids_stride1;
  const void* topk_weights;
  int32_t topk_weights_dtype;
  int64_t topk_weights_stride0, topk_weights_stride1;
  const uint8_t* is_padding; /* nullable */
  int64_t is_padding_stride0;
  uint8_t* x; /* E2M1 pairs [T, K/2] */
  int64_t x_stride0;
  int32_t* x_sf; /* packed E4M3 block scales [T, K/64] */
  int64_t x_sf_stride0;
  float* x_scales; /* [T] */
  void* shared_x;  /* nullable: bf16 [T, K] copy, or fp8 [T, K] (shared_x_dtype) */
  int64_t shared_x_stride0;
  int32_t shared_x_dtype;    /* MOE_SHARED_BF16 or MOE_SHARED_FP8 */
  uint8_t* shared_x_sf;      /* fp8 shared_x only: UE8M0 bytes [shared_x_sf_rows, K/128] */
  int64_t shared_x_sf_stride0, shared_x_sf_stride1;
  int64_t shared_x_sf_rows;
  int64_t shared_block_m;    /* > 0 iff shared_x_sf != NULL */
  int64_t* topk_idx_out;
  int64_t topk_idx_out_stride0, topk_idx_out_stride1;
  float* topk_weights_out;
  int64_t topk_weights_out_stride0, topk_weights_out_stride1;
  const int32_t* logical_to_physical; /* EPLB, as in moe_prepare_args_t */
  int64_t num_logical, map_stride;
  const int32_t* logical_replica_count;
  int32_t* expert_load;
  int64_t num_physical;
  const uint8_t* should_record;
  const int32_t* num_unpadded_tokens;
  const float* w2_global_scale; /* nullable [num_local_experts] */
  float* l2_alpha;              /* nullable [num_local_experts] */
  int64_t num_local_experts;
  float l2_activation_scale;
  uint32_t* device_status;
} moe_nvfp4_args_t;

moe_status_t moe_prepare_nvfp4_inputs(const moe_nvfp4_args_t* args, void* stream);

/* ------------------------------------------------------------------------ */
/* moe_prepare_inputs_noalloc                                                */
/*                                                                           */
/* No counterpart on the pages: an addition of this library for callers that */
/* cannot allocate device memory -- a plugin that is handed only its input   */
/* and output buffers, code running under a CUDA graph capture where its      */
/* framework forbids allocation, or a process held to a fixed device-memory  */
/* budget that must never call cudaMalloc (which can also synchronise the    */
/* device).                                                                  */
/*                                                                           */
/* Same arguments, checks and results as moe_prepare_inputs, except that the */
/* dispatch scratch comes from a fixed array of                              */
/* MOE_PREPARE_NOALLOC_SCRATCH_BYTES bytes inside the library (present on    */
/* every GPU that loads it, until the process exits); args->workspace and    */
/* args->workspace_bytes are ignored.  A problem whose                       */
/* moe_prepare_workspace_size() exceeds that size returns                    */
/* MOE_ERR_WORKSPACE before anything is enqueued.  Nothing is allocated: no  */
/* cudaMalloc/cudaFree or allocating library call.  The array's device       */
/* address is looked up on the first call made with a device current, so    */
/* make that first call before any stream capture (it is looked up again     */
/* when the device's context has changed, e.g. after cudaDeviceReset).       */
/* Every call on a device shares the one array and finds the previous call's */
/* contents there (each call clears what must start at zero); calls that may */
/* overlap on the GPU race on it and must be serialised by the caller.       */
/* ------------------------------------------------------------------------ */
#define MOE_PREPARE_NOALLOC_SCRATCH_BYTES (4u << 20)

moe_status_t moe_prepare_inputs_noalloc(const moe_prepare_args_t* args, void* stream);

/* ------------------------------------------------------------------------ */
/* moe_batched_experts                                                       */
/*                                                                           */
/* Defined by BatchedHummingGroupedExperts.apply and                         */
/* HummingExpertsBase.process_input / humming_forward / get_buffer_metas on  */
/* the page "vllm.model_executor.layers.fused_moe.experts.fused_humming_moe" */
/* (GROUPED_MASKED layout, block-FP8 input pre-quantised before dispatch,    */
/* apply_router_weight_on_input false).  For each expert e and each row      */
/* m < expert_num_tokens[e] (G = K/128, Gn = N/128):                          */
/*   h[n]   = sum_k deq(x_b[e,m,k]) * w13[e,n,k] * w13_scale[e,n/128,k/128]  */
/*            for n in [0, 2N); deq(x) = x * 2^(sf - 127) per 1x128 group;    */
/*            columns [0, N) are gate, [N, 2N) up; h is rounded to bf16.      */
/*   y[n]   = silu(h[n]) * h[N+n], silu(g) = g / (1 + exp(-g)), n < N          */
/*   y is requantised to fp8 e4m3 in 1x128 UE8M0 groups (same recipe as      */
/*   moe_prepare_inputs) into inter_q / inter_sf.                             */
/*   output[e,m,c] = bf16( sum_n deq(y_q[m,n]) * w2[e,c,n] * w2_scale[e,c/128,n/128] ).*/
/* Rows m >= expert_num_tokens[e] of output (and of inter_q) are not written.*/
/* Accumulation is fp32; weight block scales are applied per 128-wide K      */
/* slab in fp32.                                                              */
/*                                                                           */
/* Layouts: x_b [E*M_max, K] fp8, a_scale int32 [E*M_max, ceil(G/4)] packed  */
/* UE8M0 (a_scale_mode MOE_SF_UE8M0_PACKED) or fp32 [E*M_max, G] with       */
/* deq(x) = x * a_scale[row, k/128] (MOE_SF_FP32: the fp32 a1q_scale        */
/* [M, K/128] contract of process_input / get_buffer_metas; the requantised */
/* w2 input stays 1x128 UE8M0), w13 [E, 2N, K] fp8 K-major,                  */
/* w13_scale fp32 [E, 2N/128, G], w2 [E, K, N] fp8 N-major, w2_scale fp32     */
/* [E, K/128, Gn], output bf16 [E, M_max, K].  All contiguous.  Base pointers*/
/* of x_b, w13, w2, inter_q must be 16-byte aligned.                          */
/* inter_q fp8 [E*M_max, N] and inter_sf int32 [E*M_max, ceil(Gn/4)] may be  */
/* NULL, in which case they are carved from workspace13.  With stages ==     */
/* MOE_STAGE_W2 the caller supplies them (the w2 stage alone).               */
/* Contiguous layout (expert_offsets != NULL, [E+1] as written by           */
/* moe_prepare_inputs; HummingGroupedExperts.apply with expert_layout =     */
/* expert_offsets): expert e owns rows [expert_offsets[e],                  */
/* expert_offsets[e+1]) of x_b / a_scale / inter_q / inter_sf / output,     */
/* which are still E*M_max rows long (expert_offsets[E] <= E*M_max), and     */
/* its row count is not capped by M_max.                                     */
/* workspace2 holds split-K partials and tile counters.  It must be zero-    */
/* filled once when allocated; every call leaves its counters at zero again   */
/* (after a MOE_DEV_TIMEOUT, zero it before reuse).                           */
/* Errors: K % 128, N % 128 -> SHAPE; activation != SILU, a_scale_mode not   */
/* UE8M0_PACKED or FP32 -> UNSUPPORTED; short workspaces -> WORKSPACE.       */
/* ------------------------------------------------------------------------ */
typedef struct moe_experts_args {
  int64_t num_experts;           /* E */
  int64_t max_tokens_per_expert; /* M_max */
  int64_t hidden_size;           /* K, multiple of 128 */
  int64_t intermediate_size;     /* N, multiple of 128 */
  int32_t activation;            /* MOE_ACT_SILU */
  int32_t stages;                /* MOE_STAGE_* mask; 0 means MOE_STAGE_ALL */

  void* output;                       /* bf16 [E, M_max, K] */
  const void* hidden;                 /* fp8 [E*M_max, K] */
  const void* a_scale;                /* int32 [E*M_max, ceil(G/4)] */
  int32_t a_scale_mode;               /* MOE_SF_UE8M0_PACKED */
  const void* w13;                    /* fp8 [E, 2N, K] */
  const float* w13_scale;             /* [E, 2N/128, K/128] */
  const void* w2;                     /* fp8 [E, K, N] */
  const float* w2_scale;              /* [E, K/128, N/128] */
  const int32_t* expert_num_tokens;   /* [E] */
  const int32_t* expert_offsets;      /* nullable [E+1]: contiguous layout */

  void* inter_q;   /* nullable: fp8 [E*M_max, N] */
  void* inter_sf;  /* nullable: int32 [E*M_max, ceil(Gn/4)] */
  void* workspace13;
  size_t workspace13_bytes;
  void* workspace2;
  size_t workspace2_bytes;
  int64_t valid_shape_m; /* tuning hint: the routed rows this call expects, the     */
                         /* pages' estimate_local_valid_shape_m (T * k, scaled by   */
                         /* local / global experts); <= 0: this call has no token   */
                         /* count, so it assumes every row of the layout (E * M_max) */
  void* gate_up_dump;    /* nullable: bf16 [E*M_max, 2N] copy of h (debug/parity) */
  uint32_t* device_status;
} moe_experts_args_t;

moe_status_t moe_batched_experts(const moe_experts_args_t* args, void* stream);

/* Workspace bytes: which = 13 (workspace13: inter_q + inter_sf) or 2
 * (workspace2: split-K partials + tile counters for this valid_shape_m). */
size_t moe_batched_experts_workspace_size(int64_t num_experts, int64_t max_tokens_per_expert,
                                          int64_t hidden_size, int64_t intermediate_size,
                                          int64_t valid_shape_m, int which);

/* ------------------------------------------------------------------------ */
/* moe_topk_reduce                                                           */
/*                                                                           */
/* Defined by the finalize step of BatchedHummingGroupedExperts              */
/* (finalize_weight_and_reduce_impl -> TopKWeightAndReduceDelegate) and the  */
/* weighted top-k sum of moe_fused_mul_sum in HummingIndexedExperts.apply     */
/* ("...fused_moe.experts.fused_humming_moe"):                               */
/*   out[t, c] = bf16( sum_{j < k, idx[t,j] >= 0, slot[t,j] >= 0}            */
/*                     w[t,j] * expert_out[idx[t,j], slot[t,j], c] )          */
/* summed in fp32 in ascending j; tokens without a placed route get 0.       */
/* expert_out bf16 [E, M_max, K]; topk_idx int64 [T, k]; route_slot int32    */
/* [T, k]; topk_weights fp32 [T, k]; out bf16 [T, K]; all contiguous; the    */
/* expert_out and out base pointers 16-byte aligned; K % 8 == 0.             */
/* Contiguous layout (moe_unpermute of HummingGroupedExperts.apply): with    */
/* topk_idx == NULL, route_slot[t, j] is the row of expert_out itself (-1 =  */
/* unplaced), rows < num_experts * max_tokens_per_expert.                    */
/* num_valid_tokens (nullable DEVICE int32 scalar; the num_valid_tokens of   */
/* moe_fused_mul_sum in HummingIndexedExperts.apply): only tokens           */
/* t < *num_valid_tokens are written, rows past it are left untouched (a     */
/* negative value writes none).  The launch is sized by num_tokens, so a     */
/* call captured in a CUDA graph with the largest batch serves every smaller */
/* batch by updating the scalar.  NULL writes all num_tokens rows.           */
/* ------------------------------------------------------------------------ */
moe_status_t moe_topk_reduce(const void* expert_out, int64_t num_experts,
                             int64_t max_tokens_per_expert, int64_t hidden_size,
                             const int64_t* topk_idx, const int32_t* route_slot,
                             const float* topk_weights, int64_t num_tokens, int64_t top_k,
                             const int32_t* num_valid_tokens, void* out, void* stream);

/* ------------------------------------------------------------------------ */
/* moe_route                                                                 */
/*                                                                           */
/* Top-k ids and weights of router logits l[t, e], in fp32.                  */
/*   key[t, e] = l                     without a bias (both scorings are      */
/*                                     monotone in the logit);                */
/*               l + bias[e]           softmax with a bias (on the logit: a    */
/*                                     bias trained for scores goes with the  */
/*                                     next form);                            */
/*               exp(l - m)/z + bias   SOFTMAX | BIAS_ON_SCORE with a bias, the */
/*                                     sum z over all experts as below;        */
/*               1/(1+exp(-l)) + bias  sigmoid with a bias.                   */
/* An expert whose key is NaN or -inf is not selectable (a masked expert),    */
/* with BIAS_ON_SCORE neither one whose logit is.  (A sigmoid's score of a    */
/* logit of -inf is 0: with a bias such an expert is masked by the bias.)     */
/* Groups (num_groups > 1; E % num_groups == 0): a group's value is its       */
/* highest key, with a bias the sum of its two highest (a missing second     */
/* counts 0); only experts of the top_groups best groups stay selectable.    */
/* The k selectable experts of highest key are taken, in descending order;   */
/* among equal keys (of experts or groups) the lowest index comes first.     */
/*   softmax:  p_e = exp(l_e - m) / sum over all selectable-by-logit e'       */
/*             (l not NaN) of exp(l_e' - m); renormalize: the sum over the    */
/*             taken experts instead.                                        */
/*   sigmoid:  p_e = 1/(1+exp(-l_e)); renormalize: divided by the taken       */
/*             experts' sum + 1e-20.                                         */
/*   topk_weights[t, j] = scale * p_(ids[t, j]).                              */
/* Where fewer than k experts are selectable the rest of the row is id -1,   */
/* weight 0; padding tokens (is_padding[t] != 0) are -1 and 0 throughout.    */
/* topk_ids int32 or int64 [T, k], topk_weights fp32 [T, k], contiguous.     */
/* Errors: k < 1, k > E, E % num_groups, top_groups outside [1, num_groups],  */
/* k > top_groups * E / num_groups -> SHAPE; E > 1024, k > 32, num_groups >   */
/* 32 -> UNSUPPORTED.                                                        */
/*                                                                           */
/* moe_route_backward: d_logits[t, :] (the type of logits, every value        */
/* written) from d_weights fp32 [T, k] and the ids that moe_route gave: the   */
/* gradient of the formulas above with the selection held fixed.  Entries    */
/* with id < 0 (or >= E) contribute nothing.                                 */
/* ------------------------------------------------------------------------ */
typedef struct moe_route_args {
  int64_t num_tokens, num_experts, top_k;
  const void* logits; /* [T, E], inner stride 1 */
  int32_t logits_dtype;
  int64_t logits_stride0;
  const float* bias;         /* nullable [E] */
  const uint8_t* is_padding; /* nullable [T] */
  int32_t scoring;           /* MOE_SCORE_* */
  int32_t renormalize;
  float scale;
  int64_t num_groups, top_groups; /* 1, 1: no groups */
  void* topk_ids;
  int32_t topk_ids_dtype; /* MOE_IDS_* */
  float* topk_weights;
} moe_route_args_t;

moe_status_t moe_route(const moe_route_args_t* args, void* stream);

typedef struct moe_route_backward_args {
  int64_t num_tokens, num_experts, top_k;
  const void* logits;
  int32_t logits_dtype;
  int64_t logits_stride0;
  int32_t scoring;
  int32_t renormalize;
  float scale;
  const void* topk_ids; /* [T, k] contiguous, as moe_route wrote them */
  int32_t topk_ids_dtype;
  const float* d_weights; /* [T, k] contiguous */
  void* d_logits;         /* [T, E], the type of logits */
  int64_t d_logits_stride0;
} moe_route_backward_args_t;

moe_status_t moe_route_backward(const moe_route_backward_args_t* args, void* stream);

/* ------------------------------------------------------------------------ */
/* moe_sort_routes, moe_permute, moe_unpermute                               */
/*                                                                           */
/* Route (t, j) with id e = topk_ids[t, j] in [0, E) has row                  */
/*   route_row[t, j] = #routes to experts < e + #earlier routes (t', j') to e, */
/* earlier in (token, k) order; any other id gives -1 (an id >= E also sets   */
/* MOE_DEV_BAD_EXPERT).  expert_offsets[e] = #routes to experts < e, e <= E;  */
/* row_route[r] = t * k + j of row r, -1 for r >= expert_offsets[E].          */
/* topk_ids int32 or int64 [T, k]; expert_offsets int32 [E + 1]; route_row    */
/* and row_route int32 [T * k].  workspace: moe_sort_workspace_size() bytes,  */
/* 16-byte aligned, need not be cleared; it serves fewer routes as well.      */
/* E > 1024 -> UNSUPPORTED.                                                   */
/*                                                                           */
/* With `rows` [num_rows, K] in the order of the experts:                     */
/*   moe_permute             rows[route_row[t, j]] = x[t]; rows from           */
/*                           expert_offsets[E] on are written as zeros;        */
/*   moe_unpermute           out[t] = sum_j w[t, j] * rows[route_row[t, j]],    */
/*                           in fp32 in ascending j, rounded once; with        */
/*                           topk_weights = NULL every weight is 1, which is   */
/*                           the gradient of moe_permute (d_rows -> d_x);      */
/*   moe_unpermute_backward  d_rows[r(t, j)] = w[t, j] * d_out[t], rows from    */
/*                           expert_offsets[E] on zeros;                       */
/*                           d_weights[t, j] = <d_out[t], rows[r(t, j)]>, fp32. */
/* Routes with route_row outside [0, num_rows) are left out (weight gradient  */
/* 0); rows of `rows` that no route names are not read.  Tensors of one call  */
/* have one dtype (MOE_DTYPE_*), inner stride 1 and a row stride of their own; */
/* weights are fp32.  top_k > 32 -> UNSUPPORTED.                              */
/* ------------------------------------------------------------------------ */
size_t moe_sort_workspace_size(int64_t num_tokens, int64_t top_k, int64_t num_experts);

typedef struct moe_sort_args {
  int64_t num_tokens, top_k, num_experts;
  const void* topk_ids; /* [T, k] contiguous */
  int32_t topk_ids_dtype;
  int32_t* expert_offsets; /* [E + 1] */
  int32_t* route_row;      /* [T, k] */
  int32_t* row_route;      /* [T * k] */
  void* workspace;
  size_t workspace_bytes;
  uint32_t* device_status;
} moe_sort_args_t;

moe_status_t moe_sort_routes(const moe_sort_args_t* args, void* stream);

typedef struct moe_permute_args {
  int64_t num_tokens, hidden_size, top_k, num_experts, num_rows;
  int32_t dtype;
  const void* x; /* [T, K] */
  int64_t x_stride0;
  const int32_t* route_row;      /* [T, k] */
  const int32_t* expert_offsets; /* [E + 1] */
  void* rows;                    /* [num_rows, K] */
  int64_t rows_stride0;
} moe_permute_args_t;

moe_status_t moe_permute(const moe_permute_args_t* args, void* stream);

typedef struct moe_unpermute_args {
  int64_t num_tokens, hidden_size, top_k, num_rows;
  int32_t dtype;
  const void* rows; /* [num_rows, K] */
  int64_t rows_stride0;
  const int32_t* route_row;  /* [T, k] */
  const float* topk_weights; /* nullable [T, k] */
  void* out;                 /* [T, K] */
  int64_t out_stride0;
} moe_unpermute_args_t;

moe_status_t moe_unpermute(const moe_unpermute_args_t* args, void* stream);

typedef struct moe_unpermute_backward_args {
  int64_t num_tokens, hidden_size, top_k, num_experts, num_rows;
  int32_t dtype;
  const void* d_out; /* [T, K] */
  int64_t d_out_stride0;
  const void* rows; /* [num_rows, K] */
  int64_t rows_stride0;
  const int32_t* route_row;
  const float* topk_weights;
  const int32_t* expert_offsets;
  void* d_rows; /* [num_rows, K] */
  int64_t d_rows_stride0;
  float* d_weights; /* [T, k] */
} moe_unpermute_backward_args_t;

moe_status_t moe_unpermute_backward(const moe_unpermute_backward_args_t* args, void* stream);

/* ------------------------------------------------------------------------ */
/* moe_block_norm                                                            */
/*                                                                           */
/* The seam between two blocks: the residual stream x, the output z of the    */
/* block before and the input y of the block after.  In fp32, per token:      */
/*   n = z * rstd_post * (post_weight + weight_offset),                       */
/*       rstd_post = 1 / sqrt(mean(z^2) + eps)      (no post_weight: n = z)   */
/*   x_out = x + scale * gate * n                   (no z: x_out is x)        */
/*   y = x_out * rstd_pre * (pre_weight + weight_offset),                     */
/*       rstd_pre = 1 / sqrt(mean(x_out^2) + eps)                             */
/* x_out and y are rounded once each; y comes from the unrounded x_out.       */
/* z NULL: no x_out, gate or post_weight; pre_weight NULL: no y or rstd_pre.  */
/* x_out may be x itself (in place).  x, z, x_out, y and a full gate have     */
/* one dtype, inner stride 1 and row strides of their own; weights and a      */
/* channel gate are [K] of weight_dtype; a token gate is [T] of dtype.        */
/* rstd_post and rstd_pre: nullable fp32 [T], kept for the gradient.          */
/*                                                                           */
/* moe_block_norm_backward: d_x, d_z, d_gate (the gate's shape and type),     */
/* d_post_weight and d_pre_weight (weight_dtype) from d_x_out and d_y (either */
/* may be NULL: zero) and the inputs, rstd_post and rstd_pre of the forward.  */
/* Sums over tokens run in fp32 in a fixed order.  workspace:                 */
/* moe_block_norm_workspace_size() bytes, need not be cleared; it serves      */
/* fewer tokens as well.  Every output but d_x may be NULL.  Without tokens    */
/* the [K] gradients are zeros; tensors with a row a token and the workspace  */
/* may then be NULL.                                                          */
/* Errors: K > 16384 -> UNSUPPORTED.                                          */
/* ------------------------------------------------------------------------ */
typedef struct moe_block_norm_args {
  int64_t num_tokens, hidden_size;
  int32_t dtype, weight_dtype; /* MOE_DTYPE_* */
  const void* x;
  int64_t x_stride0;
  const void* z; /* nullable */
  int64_t z_stride0;
  const void* post_weight; /* nullable [K] */
  const void* gate;
  int32_t gate_kind; /* MOE_GATE_* */
  int64_t gate_stride0; /* row stride of a full gate, element stride of a token gate */
  float scale;
  const void* pre_weight; /* nullable [K] */
  float weight_offset, eps;
  void* x_out; /* iff z */
  int64_t x_out_stride0;
  void* y; /* iff pre_weight */
  int64_t y_stride0;
  float* rstd_post; /* nullable [T] */
  float* rstd_pre;  /* nullable [T] */
} moe_block_norm_args_t;

moe_status_t moe_block_norm(const moe_block_norm_args_t* args, void* stream);

typedef struct moe_block_norm_backward_args {
  int64_t num_tokens, hidden_size;
  int32_t dtype, weight_dtype;
  const void* x;
  int64_t x_stride0;
  const void* z; /* nullable */
  int64_t z_stride0;
  const void* post_weight; /* nullable */
  const void* gate;
  int32_t gate_kind;
  int64_t gate_stride0;
  float scale;
  const void* pre_weight; /* nullable */
  float weight_offset;
  const float* rstd_post; /* iff post_weight */
  const float* rstd_pre;  /* iff pre_weight */
  const void* d_x_out;    /* nullable */
  int64_t d_x_out_stride0;
  const void* d_y; /* nullable; needs pre_weight */
  int64_t d_y_stride0;
  void* d_x;
  int64_t d_x_stride0;
  void* d_z; /* nullable */
  int64_t d_z_stride0;
  void* d_gate; /* nullable */
  int64_t d_gate_stride0;
  void* d_post_weight; /* nullable [K] */
  void* d_pre_weight;  /* nullable [K] */
  void* workspace;
  size_t workspace_bytes;
} moe_block_norm_backward_args_t;

moe_status_t moe_block_norm_backward(const moe_block_norm_backward_args_t* args, void* stream);

size_t moe_block_norm_workspace_size(int64_t num_tokens, int64_t hidden_size);

/* ------------------------------------------------------------------------ */
/* moe_lora_linear                                                           */
/*                                                                           */
/*   out[t, n] = sum_k x[t, k] * weight[n, k]                                 */
/*             + lora_scale[a] * sum_r lora_b[a, n, r] * h[t, r],             */
/*   h[t, r] = sum_k x[t, k] * lora_a[a, r, k],  a = adapter_ids[t];          */
/* tokens with a < 0 (no adapter; a >= num_adapters also sets                 */
/* MOE_DEV_BAD_ADAPTER) take the first sum alone.  Sums are in fp32; scale*h  */
/* enters the second product as two values of the tensors' type, its rounding */
/* and the remainder (16 bits of bf16; of fp16 22, in steps of 2^-24 at the    */
/* smallest); of fp16, four or eight neighbouring ranks of a token with a      */
/* value above 65504, or all below 2^-14, are multiplied in fp32.  out is      */
/* rounded once.                                                              */
/* An adapter's values, non-finite ones too, reach its own tokens alone.      */
/* x [T, K] and out [T, N]: inner stride 1, row strides of their own; weight  */
/* [N, K], lora_a [S, R, K], lora_b [S, N, R] contiguous; adapter_ids int32   */
/* [T]; lora_scale fp32 [S]; bf16 or fp16.  An adapter of lower rank than R   */
/* has zero rows in lora_a.  num_adapters == 0: the projection alone.         */
/* workspace: moe_lora_workspace_size() bytes, need not be cleared; it serves */
/* every call with fewer tokens as well.                                      */
/* Errors: K % 8, R % 8, x_stride0 % 8 != 0, x, weight, lora_a, lora_b not    */
/* 16-byte aligned -> ALIGNMENT; R > 128, num_adapters > 1023, fp32 ->        */
/* UNSUPPORTED.  A GEMM wait that ran out sets MOE_DEV_TIMEOUT.               */
/* ------------------------------------------------------------------------ */
typedef struct moe_lora_args {
  int64_t num_tokens, in_features, out_features; /* T, K, N */
  int64_t num_adapters, rank;                    /* S, R */
  int32_t dtype;                                 /* MOE_DTYPE_BF16 or MOE_DTYPE_FP16 */
  const void* x;
  int64_t x_stride0;
  const void* weight;
  const void* lora_a;
  const void* lora_b;
  const int32_t* adapter_ids;
  const float* lora_scale;
  void* out;
  int64_t out_stride0;
  void* workspace;
  size_t workspace_bytes;
  uint32_t* device_status;
} moe_lora_args_t;

moe_status_t moe_lora_linear(const moe_lora_args_t* args, void* stream);

size_t moe_lora_workspace_size(int64_t num_tokens, int64_t in_features, int64_t out_features,
                               int64_t num_adapters, int64_t rank);

/* ------------------------------------------------------------------------ */
/* moe_norm_quant                                                            */
/*                                                                           */
/* The norm before a block with its output in 8 bits.  In fp32, per token:    */
/*   x_out = x + z                                (no z: x_out is x)          */
/*   y = x_out * rstd * (weight + weight_offset),                             */
/*       rstd = 1 / sqrt(mean(x_out^2) + eps)                                 */
/*   q = e4m3_rn_satfinite(y * (1 / qs)), qs of each 1x128 group of y by the   */
/*       recipe of moe_prepare_inputs (sf_mode UE8M0_PACKED or FP32).         */
/* x_out and y (nullable) are rounded once each; y comes from the unrounded   */
/* x_out and q from the unrounded y.  A last group of K % 128 columns has a    */
/* scale of its own; of packed exponents the last word is filled up with      */
/* zero bytes.  q [T, K] and q_sf (int32 [T, ceil(G/4)] or fp32 [T, G], G =    */
/* ceil(K/128)) are what moe_batched_experts takes as hidden and a_scale.     */
/* x_out may be x or z itself.  x, z, x_out and y have one dtype; rows have   */
/* inner stride 1 and a stride of their own; weight is [K] of weight_dtype.   */
/* rstd: nullable fp32 [T].  The gradient, with the rounding to 8 bits passed  */
/* straight through, is moe_block_norm_backward's (scale 1, no gate, no       */
/* post_weight, this weight as pre_weight, rstd as rstd_pre).                 */
/* Errors: K > 16384 -> UNSUPPORTED.                                          */
/* ------------------------------------------------------------------------ */
typedef struct moe_norm_quant_args {
  int64_t num_tokens, hidden_size;
  int32_t dtype, weight_dtype; /* MOE_DTYPE_* */
  const void* x;
  int64_t x_stride0;
  const void* z; /* nullable */
  int64_t z_stride0;
  const void* weight; /* [K] */
  float weight_offset, eps;
  void* x_out; /* iff z */
  int64_t x_out_stride0;
  void* y; /* nullable */
  int64_t y_stride0;
  void* q; /* fp8 [T, K] */
  int64_t q_stride0;
  void* q_sf;
  int32_t sf_mode; /* MOE_SF_UE8M0_PACKED or MOE_SF_FP32 */
  int64_t q_sf_stride0;
  float* rstd; /* nullable [T] */
} moe_norm_quant_args_t;

moe_status_t moe_norm_quant(const moe_norm_quant_args_t* args, void* stream);

/* ------------------------------------------------------------------------ */
/* moe_gated_linear                                                          */
/*                                                                           */
/* The first half of a gated feed-forward block (a shared expert's):          */
/*   g = x Wg^T, u = x Wu^T, out = act(g) * u,                                 */
/* with Wg rows [0, N) and Wu rows [N, 2N) of weight.  Sums, g, u and the      */
/* product are in fp32; out is rounded once.  gate_up (nullable) gets g in     */
/* columns [0, N) and u in [N, 2N), rounded once each, for the gradient.       */
/* x [T, K], out [T, N] and gate_up [T, 2N]: inner stride 1, row strides of     */
/* their own; weight [2N, K] contiguous; bf16 or fp16.  activation:            */
/* MOE_ACT_SILU or MOE_ACT_GELU_TANH.                                         */
/*                                                                           */
/* moe_gated_linear_backward: from d_out [T, N], the forward's x and weight and */
/* the gate_up that it wrote,                                                */
/*   d_g = d_out * u * act'(g), d_u = d_out * act(g),                          */
/*   d_x = d_g Wg + d_u Wu, d_weight = [d_g d_u]^T x  (either may be NULL);     */
/* d_g and d_u enter the products rounded to the tensors' type, sums are in    */
/* fp32 in a fixed order, results rounded once.  d_x [T, K] has a row stride   */
/* of its own, d_weight [2N, K] is contiguous.  Without tokens d_weight is     */
/* zeros; tensors with a row a token may then be NULL.  workspace:             */
/* moe_gated_linear_workspace_size() bytes, 16-byte aligned, need not be        */
/* cleared; it serves fewer tokens as well.                                   */
/* Errors: K % 8, x_stride0 % 8 != 0, x or weight not 16-byte aligned ->       */
/* ALIGNMENT; fp32, MOE_ACT_NONE -> UNSUPPORTED.  A GEMM wait that ran out      */
/* sets MOE_DEV_TIMEOUT.                                                      */
/* ------------------------------------------------------------------------ */
typedef struct moe_gated_linear_args {
  int64_t num_tokens, in_features, out_features; /* T, K, N */
  int32_t dtype;                                 /* MOE_DTYPE_BF16 or MOE_DTYPE_FP16 */
  int32_t activation;                            /* MOE_ACT_* */
  const void* x;
  int64_t x_stride0;
  const void* weight; /* [2N, K] */
  void* out;
  int64_t out_stride0;
  void* gate_up; /* nullable */
  int64_t gate_up_stride0;
  uint32_t* device_status;
} moe_gated_linear_args_t;

moe_status_t moe_gated_linear(const moe_gated_linear_args_t* args, void* stream);

typedef struct moe_gated_linear_backward_args {
  int64_t num_tokens, in_features, out_features;
  int32_t dtype;
  int32_t activation;
  const void* d_out;
  int64_t d_out_stride0;
  const void* x;
  int64_t x_stride0;
  const void* weight;
  const void* gate_up;
  int64_t gate_up_stride0;
  void* d_x; /* nullable */
  int64_t d_x_stride0;
  void* d_weight; /* nullable [2N, K] */
  void* workspace;
  size_t workspace_bytes;
  uint32_t* device_status;
} moe_gated_linear_backward_args_t;

moe_status_t moe_gated_linear_backward(const moe_gated_linear_backward_args_t* args, void* stream);

size_t moe_gated_linear_workspace_size(int64_t num_tokens, int64_t in_features,
                                       int64_t out_features);

/* ------------------------------------------------------------------------ */
/* moe_w4_linear                                                             */
/*                                                                           */
/* Products of few rows with 4-bit weights and group scales.  A matrix is      */
/*   W[n, k] = scales[n, k/G] * (q[n, k] - zeros[n, k/G])      INT4 (no zeros: */
/*             q - 8), scales of dtype, zeros uint8 (their lower four bits);   */
/*   W[n, k] = 2^(scales[n, k/G] - 127) * e2m1(q[n, k])        E2M1, scales    */
/*             uint8 (255: not a number).                                    */
/* q[n, k] is the low (k even) or high (k odd) half of byte k/2 of row n.      */
/*   topk_ids NULL:  out[t] = x[t] W^T, one matrix [N, K];                      */
/*   topk_ids [T, k]: out[t * k + j] = x[t] W_e^T of matrix e = topk_ids[t, j]  */
/*                   of [E, N, K]; other ids give a row of zeros (id >= E also  */
/*                   sets MOE_DEV_BAD_EXPERT).  With top_k 1 every row of x has */
/*                   an expert of its own, as the second product of a layer     */
/*                   needs it.                                               */
/* activation MOE_ACT_NONE: out has N columns.  Else rows [0, N/2) are a gate,  */
/* rows [N/2, N) up, and out = act(gate) * up has N/2 columns.                 */
/* A group's sum is in fp32, of exact products; the scale multiplies it there;*/
/* out is rounded once.  x enters as it is down to 2^-31 (fp16: 2^-28) of its */
/* row's largest finite value, and off by at most 2^-39 of that below.        */
/* (Scales below 2^-96 need not keep all that: the sums are subnormal.)       */
/* A matrix passes once for as many of its rows of x as a CTA has room for:   */
/* 16 at most to K = 4096, 9 at 7168, 8 at 8192, 5 at 14336, 4 at 16384, 2     */
/* above 24064; with routes in the hundreds one or two fewer.                 */
/* A row of x, non-finite values too, reaches its own rows of out alone.  x   */
/* [T, K] and out: inner stride 1, row strides of their own; weight, scales and*/
/* zeros contiguous; bf16 or fp16.                                            */
/* Errors: K % G, an odd N with an activation -> SHAPE; G other than 32, 64,  */
/* 128 (E2M1: 32), zeros with E2M1, more than 1024 rows of out (routes), E >  */
/* 1024, K > 32768, N >= 2^20, fp32 -> UNSUPPORTED; x, weight or x's rows not */
/* on 16-byte boundaries -> ALIGNMENT.                                        */
/* ------------------------------------------------------------------------ */
typedef struct moe_w4_linear_args {
  int64_t num_tokens, in_features, matrix_rows; /* T, K, N */
  int64_t num_experts, top_k;                   /* with topk_ids */
  int64_t group_size;                           /* G */
  int32_t dtype;                                /* MOE_DTYPE_BF16 or MOE_DTYPE_FP16 */
  int32_t format;                               /* MOE_W4_* */
  int32_t activation;                           /* MOE_ACT_* */
  const void* x;
  int64_t x_stride0;
  const void* weight; /* [E, N, K/2] bytes */
  const void* scales; /* [E, N, K/G] */
  const void* zeros;  /* nullable [E, N, K/G] */
  const void* topk_ids;
  int32_t topk_ids_dtype; /* MOE_IDS_* */
  void* out;
  int64_t out_stride0;
  uint32_t* device_status;
} moe_w4_linear_args_t;

moe_status_t moe_w4_linear(const moe_w4_linear_args_t* args, void* stream);

/* ------------------------------------------------------------------------ */
/* Utilities                                                                 */
/* ------------------------------------------------------------------------ */
int moe_abi_version(void);
/* Message of the last host-side error on this thread ("" if none). */
const char* moe_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_PREP_H */
