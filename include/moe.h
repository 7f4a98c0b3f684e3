/*
 * moe.h -- C ABI of libmoe: the forward pass of one Hunyuan-style
 * mixture-of-experts layer on an AMD Instinct MI355X (gfx950).
 *
 * The layer (Hy3 on CANN NPU guide, section 1 and section 8.5; Hy4-preview
 * tutorial, section 1; HunyuanImage-3.0 multi-stream article, source
 * walkthrough parts 1-3):
 *
 *   s      = sigmoid(x W_r^T + b)                         gating scores
 *   idx    = the top-k experts of each token by s          (ties: lower index;
 *                                                           a NaN s counts as 0)
 *   w      = rho * s[idx] / sum(s[idx])                    route_norm, scaling
 *   y_e    = W_d,e ( silu(W_g,e x) * (W_u,e x) )           SwiGLU expert FFN
 *   out    = sum_j w_j y_idx_j(x)  +  FFN_shared(x)        combine + shared
 *
 * computed as Gating -> InitRouting (permutation) -> grouped GEMM ->
 * FinalizeRouting (weighted combine) -> add of the always-on shared expert,
 * which runs on a second stream joined by an event where that pays (see
 * moe_layer_forward).
 *
 * Conventions for every call:
 *  - Pointers are DEVICE pointers unless marked "host".  The caller owns all
 *    memory; the library never allocates device memory after moe_ctx_create
 *    (which creates two events) and never frees caller memory.
 *  - Activations, outputs, workspaces, router weights and packed expert
 *    weights are read or written with 16-byte vector accesses and must start
 *    16-byte aligned (any allocation is); a misaligned one returns
 *    MOE_ERR_INVALID_ARG.  The sources of moe_mx_quantize, moe_fp8_quantize
 *    and moe_pack_experts and moe_permute's topk_idx may be unaligned.
 *  - Streams are hipStream_t handles passed as void* (NULL = the null stream).
 *    Calls enqueue work on the given stream and return without synchronising;
 *    results are ready when that stream reaches the point of the call.
 *  - Arguments are validated before anything is enqueued.  A failed validation
 *    returns MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED / MOE_ERR_WORKSPACE and
 *    enqueues nothing.  T == 0 returns MOE_OK and enqueues nothing; T * top_k
 *    above 2^31 - 1 (the int32 pair indices) returns MOE_ERR_UNSUPPORTED.  A HIP
 *    launch error returns MOE_ERR_DEVICE (text in moe_ctx_last_error).  Faults
 *    inside kernels surface at the caller's next synchronisation, as with any
 *    HIP library.  No call aborts or throws.
 *  - Outputs are bit-identical from run to run for identical inputs (no
 *    floating-point atomics; fixed reduction orders).
 *  - A moe_ctx may be used by one host thread at a time.
 *
 * Shape limits: 1 <= E <= 1024, 1 <= k <= min(E, 16); H a multiple of 256;
 * I and I_s multiples of 128 (256 for MX-fp8 and MXFP4); I_s = 0 means no
 * shared expert.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_API __attribute__((visibility("default")))

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1, /* null pointer, bad size, bad enum            */
  MOE_ERR_UNSUPPORTED = 2, /* valid but not implemented (dtype combination) */
  MOE_ERR_WORKSPACE = 3,   /* workspace smaller than moe_workspace_bytes() */
  MOE_ERR_DEVICE = 4       /* a HIP call failed                            */
} moe_status;

typedef enum moe_dtype {
  MOE_F32 = 0,   /* IEEE binary32                                           */
  MOE_BF16 = 1,  /* bfloat16, round-to-nearest-even on every store          */
  MOE_MXFP8 = 2, /* OCP MX: E4M3 (FN) elements, one E8M0 scale per 32       */
  MOE_MXFP4 = 3, /* OCP MX: E2M1 elements (two per byte, low nibble first),
                    one E8M0 scale per 32; expert weights only (W4A8)      */
  MOE_FP8 = 4    /* E4M3 (FN) with one static fp32 scale per tensor        */
} moe_dtype;

/* Layer description (host struct).  Field names follow HYV3Config (Hy3 guide,
 * section 1).  Supported dtype combinations (act, expert, out):
 *   (F32, F32, F32)     all-fp32 layer
 *   (BF16, BF16, BF16)  bf16 activations and experts, fp32 accumulation
 *   (BF16, MXFP8, BF16) MX-fp8 experts; activations x and the SwiGLU output
 *                       are quantised to MX-fp8 on the fly (32-element blocks
 *                       along the reduction axis); bf16 output
 *   (BF16, MXFP4, BF16) W4A8, the hybrid recipe of the Hy3 guide, section 8.2:
 *                       routed experts MXFP4 (scale X = floor(log2 max|v|) - 2,
 *                       E2M1 round-to-nearest-even, saturating at 6), the
 *                       shared expert MX-fp8 (W8A8), activations MX-fp8 as
 *                       above; bf16 output
 *   (BF16, FP8, BF16)   static per-tensor FP8 W8A8 (the FP8 checkpoints of the
 *                       Hy3 guide, section 2, and the Hy4 tutorial's w8a8
 *                       weights): every expert weight matrix has one fp32
 *                       scale max|w| / 448 (computed by moe_pack_experts);
 *                       x and h are quantised with the fixed activation
 *                       scales fp8_x_scale / fp8_h_scale / fp8_sh_h_scale;
 *                       codes are E4M3 of fp32(v / scale), round to nearest
 *                       even, saturating; products are scaled by weight scale
 *                       x activation scale after fp32 accumulation
 * The router always runs in fp32 on the unquantised x. */
typedef struct moe_desc {
  int32_t hidden;                /* H                                        */
  int32_t num_experts;           /* E routed experts                         */
  int32_t top_k;                 /* k (num_experts_per_tok)                  */
  int32_t inter;                 /* I, routed expert intermediate size       */
  int32_t shared_inter;          /* I_s, 0 = no shared expert                */
  float router_scaling_factor;   /* rho, multiplies the routed weights only  */
  int32_t route_norm;            /* 1: divide selected scores by their sum   */
  int32_t act_dtype;             /* moe_dtype of x                           */
  int32_t expert_dtype;          /* moe_dtype of the packed expert weights   */
  int32_t out_dtype;             /* moe_dtype of y, shared output and out    */
  /* static activation scales (> 0), read only when expert_dtype == MOE_FP8:
   * x (routed and shared experts), the routed SwiGLU output h, and the
   * shared expert's h */
  float fp8_x_scale, fp8_h_scale, fp8_sh_h_scale;
} moe_desc;

/* Device pointers to the layer's weights (host struct). */
typedef struct moe_weights {
  const float *router_w;           /* [E,H] fp32, row-major                 */
  const float *router_bias;        /* [E] fp32 logit bias, or NULL          */
  const void *gate_up;             /* routed gate+up, packed (moe_pack_experts) */
  const void *down;                /* routed down, packed                   */
  const uint8_t *gate_up_scale;    /* MX: packed E8M0 scales; FP8: fp32 per-tensor
                                      scales [E][2] (gate, up), down [E]; else NULL */
  const uint8_t *down_scale;
  const void *sh_gate_up;          /* shared expert, packed with shared = 1 */
  const void *sh_down;
  const uint8_t *sh_gate_up_scale;
  const uint8_t *sh_down_scale;
} moe_weights;

typedef struct moe_ctx moe_ctx;

/* Create a context on HIP device `device`.  `side_stream` (borrowed, never
 * destroyed by the library) is where moe_layer_forward runs the shared
 * expert; NULL runs it on the caller's stream.  The context owns two HIP
 * events (the input-ready and shared-done events of the HunyuanImage-3.0
 * article, source walkthrough part 3).  Returns MOE_ERR_DEVICE if the device
 * is not a gfx950 GPU. */
MOE_API moe_status moe_ctx_create(int device, void *side_stream, moe_ctx **out /* host */);
MOE_API moe_status moe_ctx_destroy(moe_ctx *ctx);

/* Static text for a status code; never NULL. */
MOE_API const char *moe_status_string(moe_status s);
/* Text of the last HIP error seen by calls on ctx ("" if none). */
MOE_API const char *moe_ctx_last_error(const moe_ctx *ctx);

/* Workspace sizes in bytes for a call with T tokens.
 * which: MOE_WS_ROUTE, MOE_WS_PERMUTE, MOE_WS_GROUPED_FFN (routed, shared=0),
 * MOE_WS_SHARED_FFN (shared=1), MOE_WS_LAYER.  0 on invalid arguments. */
enum { MOE_WS_ROUTE = 0, MOE_WS_PERMUTE = 1, MOE_WS_GROUPED_FFN = 2, MOE_WS_SHARED_FFN = 3,
       MOE_WS_LAYER = 4 };
MOE_API size_t moe_workspace_bytes(const moe_desc *desc /* host */, int32_t T, int which);

/* Packed weight sizes in bytes.  shared: 0 routed experts, 1 shared expert.
 * which: MOE_PACK_GATE_UP, MOE_PACK_DOWN, MOE_PACK_GATE_UP_SCALE,
 * MOE_PACK_DOWN_SCALE (scales are 0 bytes unless expert_dtype is MX-fp8,
 * MXFP4 or FP8; the shared expert of an MXFP4 layer is packed as MX-fp8;
 * FP8 scales are fp32, 2 per expert for gate/up and 1 for down). */
enum { MOE_PACK_GATE_UP = 0, MOE_PACK_DOWN = 1, MOE_PACK_GATE_UP_SCALE = 2,
       MOE_PACK_DOWN_SCALE = 3 };
MOE_API size_t moe_packed_bytes(const moe_desc *desc /* host */, int shared, int which);

/* Pack expert weights into the kernels' layout (the FusedMoEGMM weight of
 * the HunyuanImage-3.0 article, part 1, built from per-expert [out,in]
 * matrices).  Inputs, row-major, src_dtype MOE_F32 or MOE_BF16:
 *   gate [E,I,H], up [E,I,H], down [E,H,I]   (shared: E = 1, I = I_s)
 * Outputs in desc->expert_dtype (MX-fp8 for the shared expert of an MXFP4
 * layer): gate_up_out, down_out, and for MX formats the scale arrays
 * (quantised here: OCP MX rule, blocks of 32 along the reduction axis).
 * Sizes from moe_packed_bytes.  Layout: 4 KiB blocks of 16 output rows x 256
 * bytes of K (MXFP4: 2 KiB blocks of 16 rows x 256 K elements), ordered
 * [expert][row block][K chunk]; gate and up row blocks alternate (gate
 * block j, then up block j). */
MOE_API moe_status moe_pack_experts(const moe_desc *desc /* host */, int shared, int src_dtype,
                            const void *gate, const void *up, const void *down,
                            void *gate_up_out, void *down_out, uint8_t *gate_up_scale_out,
                            uint8_t *down_scale_out, void *stream);

/* MX-fp8 quantisation of a row-major [rows, cols] matrix along its rows
 * (cols a multiple of 32): q [rows, cols] E4M3 codes, scale [rows, cols/32]
 * E8M0 bytes.  src_dtype MOE_F32 or MOE_BF16.  OCP MX v1.0 rule: X =
 * floor(log2 max|v|) - 8 clamped to [-127, 127] (zero blocks: -127), codes
 * = E4M3 round-to-nearest-even of v / 2^X saturated to +-448. */
MOE_API moe_status moe_mx_quantize(const void *src, int src_dtype, int64_t rows, int64_t cols,
                           uint8_t *q, uint8_t *scale, void *stream);

/* Static per-tensor FP8 quantisation of n elements (n a multiple of 8):
 * q[i] = E4M3 (FN) of fp32(src[i] / scale), round to nearest even,
 * saturating to +-448.  src_dtype MOE_F32 or MOE_BF16; scale > 0 (host). */
MOE_API moe_status moe_fp8_quantize(const void *src, int src_dtype, int64_t n, float scale,
                            uint8_t *q, void *stream);

/* Gating (Hy3 guide, section 1 and section 8.5 "Gating"; HunyuanImage-3.0
 * article part 3: the gate yields expert_index and topk_weight).
 *   x [T,H] (desc->act_dtype), router_w [E,H] fp32, router_bias [E] or NULL
 *   -> topk_idx [T,k] int32, experts of each token best first,
 *      topk_w   [T,k] fp32, rho * s / sum(selected s) (route_norm = 1).
 * ws: moe_workspace_bytes(desc, T, MOE_WS_ROUTE) bytes (fp32 logits). */
MOE_API moe_status moe_route(moe_ctx *ctx, const moe_desc *desc /* host */, const void *x, int32_t T,
                     const float *router_w, const float *router_bias, int32_t *topk_idx,
                     float *topk_w, void *ws, size_t ws_bytes, void *stream);

/* InitRouting (Hy3 guide, section 8.1 "MoE EP" and section 8.5): group the
 * T*k (token, slot) pairs by expert.  Pair f = t*k + j.
 *   topk_idx [T,k] int32: every entry in [0, E), distinct within a token
 *   -> expert_counts [E], expert_offsets [E+1] (exclusive prefix, last = T*k),
 *      sorted_src [T*k]: row r -> pair f, rows of one expert in ascending f,
 *      dest [T*k]:       pair f -> row r.
 * Entries outside [0, E) or repeated within a token give an unspecified (but
 * in-bounds) permutation.  ws: moe_workspace_bytes(.., MOE_WS_PERMUTE). */
MOE_API moe_status moe_permute(moe_ctx *ctx, const moe_desc *desc /* host */, const int32_t *topk_idx,
                       int32_t T, int32_t *expert_counts, int32_t *expert_offsets,
                       int32_t *sorted_src, int32_t *dest, void *ws, size_t ws_bytes,
                       void *stream);

/* Grouped expert GEMM (Hy3 guide, sections 8.1 and 8.5 "grouped GMM";
 * HunyuanImage-3.0 article part 1, FusedMoEGMM(num_experts, hidden_size,
 * intermediate_size)): for every row r of expert e (rows [offsets[e],
 * offsets[e+1]) ), with token t = sorted_src[r] / k,
 *   y[r] = W_d,e ( silu(W_g,e x[t]) * (W_u,e x[t]) ).
 * shared = 1 runs the shared expert instead: sorted_src and expert_offsets
 * are ignored (may be NULL), rows are the T tokens, y is [T,H].
 *   x [T,H] (act_dtype), y [T*k,H] or [T,H] (out_dtype).
 * ws: moe_workspace_bytes(.., MOE_WS_GROUPED_FFN or MOE_WS_SHARED_FFN). */
MOE_API moe_status moe_grouped_ffn(moe_ctx *ctx, const moe_desc *desc /* host */,
                           const moe_weights *w /* host */, int shared, const void *x, int32_t T,
                           const int32_t *sorted_src, const int32_t *expert_offsets, void *y,
                           void *ws, size_t ws_bytes, void *stream);

/* FinalizeRouting + shared add (Hy3 guide, section 8.5; HunyuanImage-3.0
 * article part 3, output = shared-MLP output + combined output):
 *   out[t] = (sum_{j<k} topk_w[t,j] * y[dest[t*k+j]]) + shared_out[t]
 * summed in fp32 in slot order, shared_out added last (NULL: none).
 *   y [T*k,H], shared_out [T,H], out [T,H], all in out_dtype. */
MOE_API moe_status moe_combine(moe_ctx *ctx, const moe_desc *desc /* host */, const void *y,
                       const int32_t *dest, const float *topk_w, const void *shared_out, int32_t T,
                       void *out, void *stream);

/* The whole layer on `stream` (Hy3 guide, section 8.5 two-stream schedule):
 * (8-bit and MXFP4 experts: quantise x;) gating, permutation and the routed
 * gate/up GEMM on `stream`, then the input-ready event; the side stream
 * waits on it and runs the shared expert beside the routed down GEMM, then
 * records the shared-done event, which `stream` waits on before the
 * combine.  The side stream is used where the overlap was measured to pay:
 * not for a shared expert under 1 MiB of weights (launch-bound layers), and
 * not at 256 or more rows per routed expert (T * k >= 256 * E, where every
 * GEMM is bound by the matrix cores); there the shared expert runs on
 * `stream` in the same place -- for f32 / bf16 experts with I_s equal to I
 * (and fewer than 1024 experts) as one more segment of the routed grouped
 * GEMMs, whose last partial round of tiles it fills; the result is the same
 * bit for bit.  On return `stream` has been made to wait for
 * the side stream, so work queued on `stream` afterwards sees the finished
 * layer.
 *   x [T,H] (act_dtype), out [T,H] (out_dtype).
 * ws: moe_workspace_bytes(desc, T, MOE_WS_LAYER) bytes; its layout is
 * internal, except that moe_layer_ws_topk() locates the routing result. */
MOE_API moe_status moe_layer_forward(moe_ctx *ctx, const moe_desc *desc /* host */,
                             const moe_weights *w /* host */, const void *x, int32_t T, void *out,
                             void *ws, size_t ws_bytes, void *stream);

/* moe_layer_forward with x also given as codes of the experts' activation
 * format, as moe_rms_norm writes them beside y, so that the experts read those
 * and x is not quantised again: xq [T,H] E4M3; xq_scale [T,H/32] E8M0 for
 * MX-fp8 and MXFP4 experts, NULL for FP8 ones (whose codes are of
 * x / fp8_x_scale).  Gating reads x, as it does without them.  Both arrays
 * 16-byte aligned.  Layers of f32 or bf16 experts return
 * MOE_ERR_UNSUPPORTED.  Given the codes that moe_layer_forward makes
 * (moe_mx_quantize, moe_fp8_quantize) the result is the same bit for bit. */
MOE_API moe_status moe_layer_forward_quantized(moe_ctx *ctx, const moe_desc *desc /* host */,
                             const moe_weights *w /* host */, const void *x, const uint8_t *xq,
                             const uint8_t *xq_scale, int32_t T, void *out, void *ws,
                             size_t ws_bytes, void *stream);

/* Per-stage timing of moe_layer_forward.  With profiling enabled the call
 * records a pair of timing events around each stage on the stream the stage
 * runs on; moe_ctx_stage_ms then waits for the last call's events and writes
 * each stage's duration in milliseconds (0 for stages that did not run):
 *   MOE_STAGE_ROUTE, MOE_STAGE_MX_QUANT, MOE_STAGE_PERMUTE,
 *   MOE_STAGE_GATE_UP (routed gate/up GEMM + SwiGLU, one kernel),
 *   MOE_STAGE_DOWN (routed down GEMM, one kernel),
 *   MOE_STAGE_SHARED_GATE_UP, MOE_STAGE_SHARED_DOWN, MOE_STAGE_COMBINE.
 * Enabling creates the events (the only allocation after moe_ctx_create);
 * the timing adds an event record between kernels, so leave it off when the
 * layer's own latency is what is measured. */
enum { MOE_STAGE_ROUTE = 0, MOE_STAGE_MX_QUANT = 1, MOE_STAGE_PERMUTE = 2, MOE_STAGE_GATE_UP = 3,
       MOE_STAGE_DOWN = 4, MOE_STAGE_SHARED_GATE_UP = 5, MOE_STAGE_SHARED_DOWN = 6,
       MOE_STAGE_COMBINE = 7, MOE_NUM_STAGES = 8 };
MOE_API moe_status moe_ctx_set_profiling(moe_ctx *ctx, int enable);
MOE_API moe_status moe_ctx_stage_ms(moe_ctx *ctx, float *ms /* host, MOE_NUM_STAGES */);

/* Byte offsets, inside a moe_layer_forward workspace for T tokens, of the
 * topk_idx [T,k] int32 and topk_w [T,k] fp32 arrays the call wrote. */
MOE_API moe_status moe_layer_ws_topk(const moe_desc *desc /* host */, int32_t T,
                             size_t *idx_offset /* host */, size_t *w_offset /* host */);

/* moe_layer_forward with no caller workspace and no allocation, for callers
 * that cannot call hipMalloc: code under HIP graph capture, tight serving
 * loops, harnesses that forbid allocation.  The workspace is a static device
 * array of MOE_NOALLOC_SCRATCH_BYTES (64 MiB) inside the library, one copy
 * per GPU, held until the process ends; moe_ctx_create looks up its address
 * on the context's device.  Arguments and results are those of
 * moe_layer_forward.  If moe_workspace_bytes(desc, T, MOE_WS_LAYER) exceeds
 * the array the call returns MOE_ERR_WORKSPACE (text in moe_ctx_last_error)
 * and enqueues nothing; for the Hy3 shape in bf16 (H = 4096, E = 192, k = 8,
 * I = I_s = 1536) that admits up to T = 548 tokens (64 tokens use 11.5 MiB).  Every call on one GPU
 * shares the array and leaves its contents behind: calls that can overlap on
 * one GPU (other streams or contexts without ordering between them) race and
 * give undefined results.  Nothing in the array needs to start at zero. */
#define MOE_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
MOE_API moe_status moe_layer_forward_noalloc(moe_ctx *ctx, const moe_desc *desc /* host */,
                                     const moe_weights *w /* host */, const void *x, int32_t T,
                                     void *out, void *stream);

/* ---------------------------------------------------------------------------
 * Operators next to the layer: RMS norm, the paged KV cache, attention over
 * it; products in E4M3 with a scale per block of 128; norms of queries and keys
 * for each head with the rotation by position; log probabilities of tokens.
 * They need no moe_ctx; the conventions above hold (device pointers,
 * 16-byte alignment, asynchronous, arguments checked first, no allocation,
 * bit-identical results from run to run).  A call with zero rows is a no-op
 * that returns MOE_OK. */

#define MOE_NO_QUANT (-1)

/* RMS norm with the residual's addition and an output in 8 bits:
 *
 *   s = x + residual                               (fp32; s = x if NULL)
 *   y = s / sqrt(mean(s^2) + eps) * weight         (64 bits, from the unrounded s)
 *   residual_out = s, y_out = y                    (rounded once to `dtype`)
 *   q: codes of the unrounded y
 *
 * dtype: MOE_F32 or MOE_BF16, for x, residual, weight, residual_out and y.
 * Row strides are in elements, rows contiguous inside; outputs are
 * [rows][hidden] contiguous and may be the inputs if those are, too.
 * q_dtype: MOE_NO_QUANT; MOE_MXFP8 (q E4M3 [rows][hidden], q_scale E8M0
 * [rows][hidden/32], the rule of moe_mx_quantize; hidden a multiple of 32);
 * MOE_FP8 (E4M3 of y / fp8_scale in 64 bits, round to nearest even,
 * saturating: moe_fp8_quantize without its rounding to fp32).  A NaN
 * becomes the NaN code and an infinity saturates.  residual_out is NULL
 * exactly where residual is; y may be NULL with an 8-bit output.  Any
 * hidden >= 1; x, residual, weight, y and residual_out need only their
 * element's alignment (16 bytes and strides of whole 16-byte pieces are
 * faster), q 16 bytes. */
MOE_API moe_status moe_rms_norm(const void *x, int64_t x_stride, const void *residual,
                        int64_t residual_stride, const void *weight, int dtype, int32_t rows,
                        int32_t hidden, float eps, void *residual_out, void *y, int q_dtype,
                        float fp8_scale, uint8_t *q, uint8_t *q_scale, void *stream);

/* A paged KV cache (host struct): pools of pages
 * [num_pages][kv_heads][page_size][head_dim] of keys and values.
 * dtype MOE_BF16 or MOE_F32: elements; MOE_MXFP8: E4M3 codes, with E8M0
 * scale bytes [num_pages][kv_heads][page_size][head_dim/32].  page_size: a
 * power of two up to 65536; kv_heads up to 1024; head_dim 64, 128 or 256;
 * num_pages * kv_heads * page_size below 2^32 - 1.  Activations are bf16 (fp32
 * for a MOE_F32 cache). */
typedef struct moe_kv_cache {
  void *k, *v;
  uint8_t *k_scale, *v_scale;    /* MOE_MXFP8 only */
  int32_t num_pages, page_size, kv_heads, head_dim, dtype;
} moe_kv_cache;

/* One batch of new tokens (host struct; the arrays are on the device).  The
 * rows row_offsets[s] .. row_offsets[s+1] - 1 of the activations are the last
 * tokens of sequence s, whose length is kv_len[s] with them; row r is
 * position kv_len[s] - row_offsets[s+1] + r, and position p lies in slot
 * p % page_size of page page_table[s][p / page_size].  Entries that are not a
 * page (negative, or num_pages and above) hold no token.  max_rows: at least
 * the largest number of new tokens of one sequence (the rows of a sequence past
 * max_rows are not computed).  The arrays are read when
 * the calls run, so a captured graph follows lengths that change; whatever
 * they hold, no access leaves the pools and the activations.
 * max_pages * page_size + rows is at most 2^31 - 4097. */
typedef struct moe_kv_batch {
  const int32_t *page_table;     /* [seqs][max_pages] */
  const int32_t *row_offsets;    /* [seqs + 1], ascending */
  const int32_t *kv_len;         /* [seqs] */
  int32_t seqs, max_pages, rows, max_rows;
} moe_kv_batch;

/* Write the new tokens' keys and values ([rows][kv_heads][head_dim]; row and
 * head strides in elements, multiples of 16 bytes unless there is only one row
 * or head) into their pages, quantised to MX-fp8 where the cache is (the rule of
 * moe_mx_quantize over head_dim; a NaN becomes the NaN code).  Rows of no
 * sequence or page are dropped.  moe_kv_read is the way back: k, v
 * [rows][kv_heads][head_dim] contiguous, dequantised and rounded once; zeros
 * for rows of no sequence or page. */
MOE_API moe_status moe_kv_write(const moe_kv_cache *cache /* host */, const moe_kv_batch *batch /* host */,
                        const void *k, int64_t k_row, int64_t k_head, const void *v,
                        int64_t v_row, int64_t v_head, void *stream);
MOE_API moe_status moe_kv_read(const moe_kv_cache *cache /* host */, const moe_kv_batch *batch /* host */,
                       void *k, void *v, void *stream);

/* Attention of the batch's rows over their sequences in the cache (the new
 * tokens' keys and values written before):
 *
 *   out[r, h] = sum_j softmax_j(scale q[r, h] . k[j, g(h)]) v[j, g(h)],
 *   g(h) = h / (heads / kv_heads),
 *
 * over the keys j <= pos(r); with window > 0 also j > pos(r) - window or
 * j < sinks.  A row that sees no key (or belongs to no sequence) gives zeros;
 * what slots hold that a row does not see, NaN included, does not reach it.  q: [rows][heads][head_dim], row and head strides in
 * elements, as above; out: [rows][heads][head_dim] contiguous.
 * Products of bf16 operands (MX-fp8 keys and values are exact in bf16) or
 * fp32 ones, accumulated in fp32; softmax statistics in fp32; with a bf16 or
 * MX-fp8 cache the softmax weights are rounded to bf16 before they multiply
 * the values.  Batches of more units (sequences x KV heads x their tiles of
 * rows) than one launch or 32-bit counts hold, some millions, return
 * MOE_ERR_UNSUPPORTED.  ws: moe_attention_workspace_bytes() bytes (0: none
 * needed, or invalid arguments), its contents need not outlive the call's
 * kernels. */
MOE_API size_t moe_attention_workspace_bytes(const moe_kv_cache *cache /* host */,
                                     const moe_kv_batch *batch /* host */, int32_t heads,
                                     int32_t window, int32_t sinks);
MOE_API moe_status moe_attention(const moe_kv_cache *cache /* host */, const moe_kv_batch *batch /* host */,
                         const void *q, int64_t q_row, int64_t q_head, int32_t heads, float scale,
                         int32_t window, int32_t sinks, void *out, void *ws, size_t ws_bytes,
                         void *stream);

/* Norms of queries and keys for each head, and their rotation by position:
 *
 *   n = x / sqrt(mean(x^2) + eps) * weight                    (over one head)
 *   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = position * inv_freq[i],
 *
 * for the pairs i < rotary_dim / 2 of elements (i, i + rotary_dim / 2), or with
 * `interleaved` the neighbours (2i, 2i + 1); elements from rotary_dim on are
 * normed only.  With norm_after the rotation comes first (the weight then
 * multiplies what is turned already; the mean is the same).  Angles are held in 64 bits,
 * sines and cosines rounded to fp32, the rest is fp32; one rounding to the output.
 *
 * dtype: MOE_F32 or MOE_BF16 of q, k, v, the weights [head_dim] and the outputs.
 * head_dim 64, 128 or 256; rotary_dim from 2 to head_dim, even, without
 * `interleaved` a multiple of 16.  inv_freq: [rotary_dim / 2] fp64. */
typedef struct moe_head_norm {
  const void *q_weight, *k_weight;
  const double *inv_freq;
  int32_t head_dim, rotary_dim, interleaved, norm_after, dtype;
  float eps;
} moe_head_norm;

/* q: [rows][heads][head_dim], k: [rows][kv_heads][head_dim], row and head strides
 * as for moe_kv_write; positions [rows].  q_out, k_out: contiguous, of the same
 * shapes. */
MOE_API moe_status moe_head_norm_rope(const moe_head_norm *norm /* host */, const void *q, int64_t q_row,
                              int64_t q_head, int32_t heads, const void *k, int64_t k_row,
                              int64_t k_head, int32_t kv_heads, const int32_t *positions,
                              int32_t rows, void *q_out, void *k_out, void *stream);
/* The same for the rows of a batch at their positions, with the turned keys and the
 * values v written into the cache, as moe_kv_write would (an MX-fp8 cache takes
 * the codes of the keys from 64 bits, not from their rounding to bf16).  q_out: zeros for rows of no sequence,
 * before its start or past its table; keys and values of rows without a page are
 * dropped.  The norm's dtype is that of the cache's activations, its head_dim the
 * cache's. */
MOE_API moe_status moe_head_norm_rope_write(const moe_head_norm *norm /* host */, const moe_kv_cache *cache /* host */,
                                    const moe_kv_batch *batch /* host */, const void *q,
                                    int64_t q_row, int64_t q_head, int32_t heads, const void *k,
                                    int64_t k_row, int64_t k_head, const void *v, int64_t v_row,
                                    int64_t v_head, void *q_out, void *stream);

/* Product of activations [rows, k] with weights [n, k] in E4M3, fp32 scales: one
 * per row and 128 columns of the activations, one per 128 x 128 of the weights (the
 * last blocks may be smaller):
 *
 *   y[r][j] = sum_b x_scale[r][b] w_scale[j / 128][b] sum_{c in block b} xq[r][c] wq[j][c]
 *
 * rounded once.  The product of both scales and all sums are fp32.  A block's scale is
 * max|v| times the fp32 number 1/448 (not max|v| / 448, which may differ by a step), rounded to
 * fp32, at least 2^-126, 0 for zeros; its codes are E4M3 of v / scale (the exact quotient,
 * round to nearest even, saturating).  A block with an infinity or NaN gets a NaN scale
 * and NaN codes, which make every sum they enter NaN.
 *
 * Codes are kept packed: blocks of 16 rows x 128 columns, 2048 bytes,
 * [rows / 16][cols / 128], both counts rounded up and filled with zeros; in a block
 * byte 1024 h + 16 l + i holds row l % 16, column 32 (l / 16) + 16 h + i.
 * moe_block_packed_bytes: their size (0: invalid).  Activation scales are
 * [cols / 128][rows rounded up to 16], weight scales [n / 128][k / 128].
 * rows, n, k up to 2^30. */
MOE_API size_t moe_block_packed_bytes(int32_t rows, int32_t cols);
/* Activations x (MOE_F32 or MOE_BF16, an element's alignment, any row stride) to
 * packed codes and scales. */
MOE_API moe_status moe_block_quantize(const void *x, int dtype, int64_t row_stride, int32_t rows, int32_t cols,
                              uint8_t *q, float *scale, void *stream);
/* Weights to packed codes: MOE_F32 or MOE_BF16 are quantised, their scales written;
 * MOE_FP8 are E4M3 codes already (with scales of the caller's; scale is not
 * used). */
MOE_API moe_status moe_block_pack(const void *w, int dtype, int64_t row_stride, int32_t n, int32_t k,
                          uint8_t *q, float *scale, void *stream);
/* out [rows][n] contiguous, MOE_F32 or MOE_BF16.  x (MOE_F32 or MOE_BF16) is
 * quantised into ws first; with xq and xq_scale (of moe_block_quantize) x is
 * not used.  ws: moe_block_linear_workspace_bytes() bytes (codes: whether xq is
 * given; 0: none needed, or invalid arguments). */
MOE_API size_t moe_block_linear_workspace_bytes(int32_t rows, int32_t n, int32_t k, int32_t codes);
MOE_API moe_status moe_block_linear(const uint8_t *wq, const float *w_scale, int32_t n, int32_t k,
                            const void *x, int x_dtype, int64_t x_stride, const uint8_t *xq,
                            const float *xq_scale, int32_t rows, void *out, int out_dtype,
                            void *ws, size_t ws_bytes, void *stream);

/* Log probabilities of given tokens, with the entropy of their distribution and its
 * best alternatives, from rows of logits (MOE_F32 or MOE_BF16; row stride in elements,
 * any alignment of an element):
 *
 *   logprob[r] = x[r][tokens[r]] - log sum_j e^x[r][j],   entropy[r] = -sum_j p_j log p_j
 *   top_token[r][0 .. top - 1]: the tokens of the largest logits, in descending order,
 *   equal ones by their index; top_logprob: theirs.
 *
 * Logits of -infinity have no part in it and the log probability -infinity, as has a
 * token outside [0, vocab).  A row of nothing else gives -infinity everywhere
 * and the entropy 0, one with a NaN or +infinity NaN; among the alternatives
 * NaN come last.  tokens: 4 or 8 bytes each (token_bytes).  top: 0 (top_logprob and
 * top_token are not used) to min(vocab, 64).  Sums in fp32. */
#define MOE_LOGPROBS_MAX_TOP 64
MOE_API moe_status moe_token_logprobs(const void *logits, int dtype, int64_t row_stride, const void *tokens,
                              int32_t token_bytes, int32_t rows, int32_t vocab, int32_t top,
                              float *logprob, float *entropy, float *top_logprob,
                              int32_t *top_token, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
