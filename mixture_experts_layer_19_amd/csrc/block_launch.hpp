// block_launch.hpp -- host-side launchers of the operators around the MoE
// layer: RMS norm, the paged KV cache, attention over it, the block-scaled 8-bit
// product, head norms with rotation, token log probabilities (internal).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// Workgroups of `threads` that one launch holds: past 2^32 threads it would run
// part of them, without an error.
constexpr long long max_groups(int threads) { return (1ll << 32) / threads - 1; }

// Row strides are in elements.  Null pointers: residual / residual_out (no
// residual), y (8-bit output only), q and q_scale (no 8-bit output).
struct NormArgs {
  const void *x, *residual, *weight;
  long long x_stride, residual_stride;
  int rows, hidden;
  float eps, fp8_scale;
  void *residual_out, *y;      // [rows][hidden]
  uint8_t *q, *q_scale;        // [rows][hidden], [rows][hidden / 32]
};
// q_fmt: FMT_MX8, FMT_FP8 or -1 (no 8-bit output).
hipError_t launch_rms_norm(const NormArgs &n, int is_bf16, int q_fmt, hipStream_t stream);

// The pool of pages [num_pages][kv_heads][page][head_dim] and one batch's
// view of it.  fmt: FMT_F32, FMT_BF16 or FMT_MX8.
struct KvArgs {
  uint8_t *k, *v, *k_scale, *v_scale;
  int num_pages, page_shift, kv_heads, head_dim, fmt;
  const int32_t *table;        // [seqs][max_pages]
  const int32_t *offsets;      // [seqs + 1]
  const int32_t *kv_len;       // [seqs]
  int seqs, max_pages, rows, max_rows;
};

// k, v: [rows][kv_heads][head_dim] with the given row and head strides (elements).
hipError_t launch_kv_write(const KvArgs &c, const void *k, const void *v, long long k_row,
                           long long k_head, long long v_row, long long v_head,
                           hipStream_t stream);
hipError_t launch_kv_read(const KvArgs &c, void *k, void *v, hipStream_t stream);

struct AttnArgs {
  KvArgs c;
  const void *q;               // [rows][heads][head_dim], strides in elements
  long long q_row, q_head;
  int heads, group;            // group = heads / kv_heads
  float scale;                 // > 0, times log2(e): the softmax runs on powers of two
  uint32_t q_sign;             // xor of every 32-bit word of q: the sign of a negative scale
  int window, sinks;           // window 0: none
  void *out;                   // [rows][heads][head_dim]
  float *part;                 // workspace: partial results of split units
  int grid;                    // workgroups of the launch
};
// Few query rows a sequence (attn_rows.hip), and many (attn_tile.hip).
// Workspace bytes (0: none needed); whether the batch is within the kernels'
// 32-bit counts.
size_t attn_rows_ws_bytes(const AttnArgs &a);
bool attn_rows_fits(const AttnArgs &a);
hipError_t launch_attn_rows(const AttnArgs &a, hipStream_t stream);
size_t attn_tile_ws_bytes(const AttnArgs &a);
bool attn_tile_fits(const AttnArgs &a);
hipError_t launch_attn_tile(const AttnArgs &a, hipStream_t stream);

// Head norms and rotation (rotate.hip).  Strides in elements.  With positions: keys to
// k_out; without: rows, positions and places are those of c's batch, keys and values go
// into its pool.
struct RotateArgs {
  KvArgs c;                    // rows, kv_heads, head_dim (and with a cache all of it)
  const void *q, *k, *v;
  long long q_row, q_head, k_row, k_head, v_row, v_head;
  const void *q_weight, *k_weight;             // [head_dim]
  const double *inv_freq;                      // [rotary / 2]
  const int32_t *positions;                    // [rows]
  int heads, rotary, interleaved, after;       // after: the weight multiplies what is turned already
  float eps;
  void *q_out, *k_out;                         // contiguous
};
hipError_t launch_rotate(const RotateArgs &a, int is_bf16, int into_cache, hipStream_t stream);

// The block-scaled E4M3 product (linear.hip).  Codes of both sides in the packed order,
// [rows / 16][k / 128] blocks of 2 KiB.
struct LinearArgs {
  const uint8_t *q;            // activations
  const float *q_scale;        // [k / 128][rows, up to a multiple of 16]
  const uint8_t *w;
  const float *w_scale;        // [n / 128][k / 128]
  void *out;                   // [rows][n]
  int rows, n, k;
  float *part;                 // splits > 1: fp32 sums [splits][rows][n up to a multiple of 4]
  int splits;                  // linear_splits of the sizes
};
hipError_t launch_block_quantize(const void *x, long long stride, int is_bf16, int rows, int cols, uint8_t *q,
                                 float *scale, hipStream_t stream);
// src: FMT_F32, FMT_BF16 (scales are written) or FMT_FP8 (codes, which only change places).
hipError_t launch_block_pack(const void *w, long long stride, int src, int n, int cols, uint8_t *q, float *scale,
                             hipStream_t stream);
// These read the sizes alone.
int linear_splits(const LinearArgs &a);
size_t linear_part_bytes(const LinearArgs &a);   // workspace of the splits (0: none)
bool linear_fits(const LinearArgs &a);           // within one launch's workgroups
bool linear_fuses(const LinearArgs &a);          // whether launch_linear_fused is the one for activations without codes
hipError_t launch_linear_fused(const LinearArgs &a, const void *x, long long stride, int is_bf16, int f32_out,
                               hipStream_t stream);
hipError_t launch_linear(const LinearArgs &a, int f32_out, hipStream_t stream);

// Token log probabilities (logprobs.hip).
constexpr int kLogprobTop = 64;                  // alternatives at most
struct LogprobArgs {
  const void *logits;          // [rows][vocab], stride in elements
  long long stride;
  const void *tokens;          // [rows] of token_bytes
  int is_bf16, token_bytes, rows, vocab, top;
  float *logprob, *entropy;    // [rows]
  float *top_logprob;          // [rows][top]
  int32_t *top_token;
};
hipError_t launch_logprobs(const LogprobArgs &a, hipStream_t stream);

}  // namespace moe
