// block_abi.hip -- the C ABI of the operators next to the MoE layer (declared
// in include/moe.h): argument checks, then the launches.
#include <math.h>

#include "../../include/moe.h"
#include "block_common.hpp"

namespace {

using namespace moe;

inline bool al(const void *p, int bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

moe_status done(hipError_t err) { return err == hipSuccess ? MOE_OK : MOE_ERR_DEVICE; }

int shift_of(int page_size) {
  for (int s = 0; s <= 16; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// Check a cache and a batch and put them in the kernels' form.
moe_status kv_args(const moe_kv_cache *c, const moe_kv_batch *b, KvArgs *o) {
  if (!c || !b) return MOE_ERR_INVALID_ARG;
  if (c->dtype < MOE_F32 || c->dtype > MOE_FP8) return MOE_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->page_size <= 0 || c->kv_heads <= 0 || c->kv_heads > 1024 ||
      c->head_dim <= 0)
    return MOE_ERR_INVALID_ARG;
  if (b->seqs < 0 || b->max_pages < 0 || b->rows < 0 || b->max_rows < 0) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16 && c->dtype != MOE_MXFP8) return MOE_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_UNSUPPORTED;
  o->page_shift = shift_of(c->page_size);
  if (o->page_shift < 0) return MOE_ERR_UNSUPPORTED;
  // positions, and those of a tile past the last key, are int32
  if (((long long)b->max_pages << o->page_shift) + b->rows > INT32_MAX - 4096) return MOE_ERR_UNSUPPORTED;
  if ((unsigned long long)c->num_pages * c->kv_heads * c->page_size >= 0xFFFFFFFFull)
    return MOE_ERR_UNSUPPORTED;
  o->fmt = c->dtype == MOE_F32 ? FMT_F32 : c->dtype == MOE_BF16 ? FMT_BF16 : FMT_MX8;
  o->k = (uint8_t *)c->k;
  o->v = (uint8_t *)c->v;
  o->k_scale = c->k_scale;
  o->v_scale = c->v_scale;
  o->num_pages = c->num_pages;
  o->kv_heads = c->kv_heads;
  o->head_dim = c->head_dim;
  o->table = b->page_table;
  o->offsets = b->row_offsets;
  o->kv_len = b->kv_len;
  o->seqs = b->seqs;
  o->max_pages = b->max_pages;
  o->rows = b->rows;
  o->max_rows = b->max_rows < b->rows ? b->max_rows : b->rows;
  if (b->rows == 0) return MOE_OK;
  if (b->seqs == 0 || b->max_rows == 0 || b->max_pages == 0) return MOE_ERR_INVALID_ARG;
  if (!c->k || !c->v || !b->page_table || !b->row_offsets || !b->kv_len) return MOE_ERR_INVALID_ARG;
  if (!al(c->k, 16) || !al(c->v, 16) || !al(b->page_table, 4) || !al(b->row_offsets, 4) ||
      !al(b->kv_len, 4))
    return MOE_ERR_INVALID_ARG;
  if (c->dtype == MOE_MXFP8 &&
      (!c->k_scale || !c->v_scale || !al(c->k_scale, 16) || !al(c->v_scale, 16)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Strides in elements of a [rows][heads][head_dim] operand of the cache's
// activation type: whole 16-byte pieces, along axes of more than one.
bool strides_ok(const KvArgs &c, int heads, int64_t row, int64_t head) {
  const int e = c.fmt == FMT_F32 ? 4 : 8;
  return (c.rows == 1 || row % e == 0) && (heads == 1 || head % e == 0);
}

moe_status attn_args(const moe_kv_cache *cache, const moe_kv_batch *batch, int heads, int window,
                     int sinks, AttnArgs *a) {
  moe_status st = kv_args(cache, batch, &a->c);
  if (st != MOE_OK) return st;
  if (heads <= 0 || heads % cache->kv_heads || window < 0 || sinks < 0) return MOE_ERR_INVALID_ARG;
  if ((long long)a->c.rows * heads > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  a->heads = heads;
  a->group = heads / cache->kv_heads;
  // a window or sinks that cover the table hide nothing
  const long long tokens = (long long)a->c.max_pages << a->c.page_shift;
  if (window >= tokens || sinks >= tokens) window = 0;
  a->window = window;
  a->sinks = window ? sinks : 0;
  return MOE_OK;
}

// Which kernel: up to 32 rows (tokens x heads of a group) a sequence fit the
// row kernel's tile, which reads the keys once and is bound by that.  So go
// fp32 with head_dim 256, whose two tiles of keys and values would not fit the
// LDS, and pages of fewer than 8 keys, which a wave's load would straddle.
bool few_rows(const AttnArgs &a) {
  return (long long)a.c.max_rows * a.group <= 32 || (a.c.fmt == FMT_F32 && a.c.head_dim == 256) || a.c.page_shift < 3;
}

constexpr int32_t kMostBlocked = 1 << 30;       // rows and columns of a block-scaled matrix

bool float_type(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16; }
bool blocked(int32_t n) { return n > 0 && n <= kMostBlocked; }
int64_t blocks_of(int64_t n) { return (n + 127) / 128; }
int64_t rows16(int64_t n) { return (n + 15) / 16 * 16; }
size_t scale_bytes(int32_t rows, int32_t cols) { return (size_t)(blocks_of(cols) * rows16(rows) * 4); }

// Check what both head norms take and put it in the kernel's form (a.c.rows,
// kv_heads and head_dim are set before).
moe_status head_norm_args(const moe_head_norm *n, int heads, const void *q, int64_t q_row, int64_t q_head,
                          const void *k, int64_t k_row, int64_t k_head, const void *q_out, RotateArgs *a) {
  if (!float_type(n->dtype) || heads <= 0 || !(n->eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if (n->rotary_dim < 2 || n->rotary_dim > n->head_dim || n->rotary_dim % (n->interleaved ? 2 : 16))
    return MOE_ERR_INVALID_ARG;
  if (n->head_dim != 64 && n->head_dim != 128 && n->head_dim != 256) return MOE_ERR_UNSUPPORTED;
  if (heads > 65536) return MOE_ERR_UNSUPPORTED;
  if (a->c.rows == 0) return MOE_OK;
  for (const void *p : {n->q_weight, n->k_weight, q, k, q_out})
    if (!p || !al(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!n->inv_freq || !al(n->inv_freq, 8)) return MOE_ERR_INVALID_ARG;
  a->c.fmt = n->dtype == MOE_F32 ? FMT_F32 : a->c.fmt == FMT_MX8 ? FMT_MX8 : FMT_BF16;
  if (!strides_ok(a->c, heads, q_row, q_head) || !strides_ok(a->c, a->c.kv_heads, k_row, k_head))
    return MOE_ERR_INVALID_ARG;
  a->q = q;
  a->k = k;
  a->q_row = q_row;
  a->q_head = q_head;
  a->k_row = k_row;
  a->k_head = k_head;
  a->q_weight = n->q_weight;
  a->k_weight = n->k_weight;
  a->inv_freq = n->inv_freq;
  a->heads = heads;
  a->rotary = n->rotary_dim;
  a->interleaved = n->interleaved != 0;
  a->after = n->norm_after != 0;
  a->eps = n->eps;
  a->q_out = const_cast<void *>(q_out);
  return MOE_OK;
}

bool logprob_args(int dtype, int32_t rows, int32_t vocab, int32_t top) {
  return float_type(dtype) && rows >= 0 && vocab > 0 && top >= 0 && top <= kLogprobTop && top <= vocab;
}
size_t workspace(const AttnArgs &a) {
  if (a.c.rows <= 0) return 0;
  return few_rows(a) ? attn_rows_ws_bytes(a) : attn_tile_ws_bytes(a);
}

}  // namespace

extern "C" {

moe_status moe_rms_norm(const void *x, int64_t x_stride, const void *residual,
                        int64_t residual_stride, const void *weight, int dtype, int32_t rows,
                        int32_t hidden, float eps, void *residual_out, void *y, int q_dtype,
                        float fp8_scale, uint8_t *q, uint8_t *q_scale, void *stream) {
  if (rows < 0 || hidden <= 0 || !(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (q_dtype != MOE_NO_QUANT && q_dtype != MOE_MXFP8 && q_dtype != MOE_FP8) return MOE_ERR_INVALID_ARG;
  if (q_dtype == MOE_MXFP8 && hidden % 32) return MOE_ERR_INVALID_ARG;
  if (q_dtype == MOE_FP8 && !(fp8_scale > 0.0f && fp8_scale < 3.0e38f)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !weight || !residual != !residual_out) return MOE_ERR_INVALID_ARG;
  if (q_dtype == MOE_NO_QUANT ? !y : !q || !al(q, 16)) return MOE_ERR_INVALID_ARG;
  if (q_dtype == MOE_MXFP8 && !q_scale) return MOE_ERR_INVALID_ARG;
  const int e = dtype == MOE_F32 ? 4 : 2;
  for (const void *p : {x, residual, weight, (const void *)residual_out, (const void *)y})
    if (!al(p, e)) return MOE_ERR_INVALID_ARG;
  const NormArgs n = {x, residual, weight, x_stride, residual ? residual_stride : 0, rows, hidden,
                      eps, fp8_scale, residual_out, y, q, q_scale};
  const int fmt = q_dtype == MOE_MXFP8 ? FMT_MX8 : q_dtype == MOE_FP8 ? FMT_FP8 : -1;
  return done(launch_rms_norm(n, dtype == MOE_BF16, fmt, (hipStream_t)stream));
}

moe_status moe_kv_write(const moe_kv_cache *cache, const moe_kv_batch *batch, const void *k,
                        int64_t k_row, int64_t k_head, const void *v, int64_t v_row,
                        int64_t v_head, void *stream) {
  KvArgs c;
  moe_status st = kv_args(cache, batch, &c);
  if (st != MOE_OK || c.rows == 0) return st;
  if (!k || !v || !al(k, 16) || !al(v, 16) || !strides_ok(c, c.kv_heads, k_row, k_head) ||
      !strides_ok(c, c.kv_heads, v_row, v_head))
    return MOE_ERR_INVALID_ARG;
  return done(launch_kv_write(c, k, v, k_row, k_head, v_row, v_head, (hipStream_t)stream));
}

moe_status moe_kv_read(const moe_kv_cache *cache, const moe_kv_batch *batch, void *k, void *v,
                       void *stream) {
  KvArgs c;
  moe_status st = kv_args(cache, batch, &c);
  if (st != MOE_OK || c.rows == 0) return st;
  if (!k || !v || !al(k, 16) || !al(v, 16)) return MOE_ERR_INVALID_ARG;
  return done(launch_kv_read(c, k, v, (hipStream_t)stream));
}

size_t moe_attention_workspace_bytes(const moe_kv_cache *cache, const moe_kv_batch *batch,
                                     int32_t heads, int32_t window, int32_t sinks) {
  AttnArgs a;
  if (attn_args(cache, batch, heads, window, sinks, &a) != MOE_OK) return 0;
  return workspace(a);
}

moe_status moe_attention(const moe_kv_cache *cache, const moe_kv_batch *batch, const void *q,
                         int64_t q_row, int64_t q_head, int32_t heads, float scale, int32_t window,
                         int32_t sinks, void *out, void *ws, size_t ws_bytes, void *stream) {
  AttnArgs a;
  moe_status st = attn_args(cache, batch, heads, window, sinks, &a);
  if (st != MOE_OK) return st;
  if (!(scale - scale == 0.0f)) return MOE_ERR_INVALID_ARG;      // infinite or NaN
  if (a.c.rows == 0) return MOE_OK;
  if (!q || !out || !al(q, 16) || !al(out, 16) || !al(ws, 16) || !strides_ok(a.c, heads, q_row, q_head))
    return MOE_ERR_INVALID_ARG;
  const size_t need = workspace(a);
  if (!(few_rows(a) ? attn_rows_fits(a) : attn_tile_fits(a))) return MOE_ERR_UNSUPPORTED;
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  a.q = q;
  a.q_row = q_row;
  a.q_head = q_head;
  // the kernels take maxima of unscaled scores, so the scale's sign goes into q; zero
  // times a masked score's -inf would be NaN, so a zero scale becomes the smallest
  // that is not (2^-149 times any score is below 2^-21), and an infinite product
  // with log2(e) the largest (whose scores, but zero, are as far apart)
  a.q_sign = scale < 0.0f ? (a.c.fmt == FMT_F32 ? 0x80000000u : 0x80008000u) : 0u;
  a.scale = fminf(fmaxf(fabsf(scale) * 1.44269504088896340736f, 0x1p-149f), 0x1.fffffep127f);
  a.out = out;
  a.part = (float *)ws;
  a.grid = 0;
  const hipStream_t s = (hipStream_t)stream;
  return done(few_rows(a) ? launch_attn_rows(a, s) : launch_attn_tile(a, s));
}

moe_status moe_head_norm_rope(const moe_head_norm *norm, const void *q, int64_t q_row, int64_t q_head,
                              int32_t heads, const void *k, int64_t k_row, int64_t k_head,
                              int32_t kv_heads, const int32_t *positions, int32_t rows, void *q_out,
                              void *k_out, void *stream) {
  if (!norm || rows < 0 || kv_heads <= 0) return MOE_ERR_INVALID_ARG;
  if (kv_heads > 1024) return MOE_ERR_UNSUPPORTED;
  RotateArgs a = {};
  a.c.rows = rows;
  a.c.kv_heads = kv_heads;
  a.c.head_dim = norm->head_dim;
  moe_status st = head_norm_args(norm, heads, q, q_row, q_head, k, k_row, k_head, q_out, &a);
  if (st != MOE_OK || rows == 0) return st;
  if (!positions || !al(positions, 4) || !k_out || !al(k_out, 16)) return MOE_ERR_INVALID_ARG;
  a.positions = positions;
  a.k_out = k_out;
  return done(launch_rotate(a, norm->dtype == MOE_BF16, 0, (hipStream_t)stream));
}

moe_status moe_head_norm_rope_write(const moe_head_norm *norm, const moe_kv_cache *cache,
                                    const moe_kv_batch *batch, const void *q, int64_t q_row,
                                    int64_t q_head, int32_t heads, const void *k, int64_t k_row,
                                    int64_t k_head, const void *v, int64_t v_row, int64_t v_head,
                                    void *q_out, void *stream) {
  if (!norm) return MOE_ERR_INVALID_ARG;
  RotateArgs a = {};
  moe_status st = kv_args(cache, batch, &a.c);
  if (st != MOE_OK) return st;
  if (norm->head_dim != cache->head_dim || norm->dtype != (cache->dtype == MOE_F32 ? MOE_F32 : MOE_BF16))
    return MOE_ERR_INVALID_ARG;
  st = head_norm_args(norm, heads, q, q_row, q_head, k, k_row, k_head, q_out, &a);
  if (st != MOE_OK || a.c.rows == 0) return st;
  if (!v || !al(v, 16) || !strides_ok(a.c, a.c.kv_heads, v_row, v_head)) return MOE_ERR_INVALID_ARG;
  a.v = v;
  a.v_row = v_row;
  a.v_head = v_head;
  return done(launch_rotate(a, norm->dtype == MOE_BF16, 1, (hipStream_t)stream));
}

size_t moe_block_packed_bytes(int32_t rows, int32_t cols) {
  return blocked(rows) && blocked(cols) ? (size_t)(rows16(rows) * blocks_of(cols) * 128) : 0;
}

moe_status moe_block_quantize(const void *x, int dtype, int64_t row_stride, int32_t rows, int32_t cols,
                              uint8_t *q, float *scale, void *stream) {
  if (!float_type(dtype) || rows < 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
  if (rows > kMostBlocked || cols > kMostBlocked) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !al(x, dtype == MOE_F32 ? 4 : 2) || !q || !al(q, 16) || !scale || !al(scale, 16))
    return MOE_ERR_INVALID_ARG;
  return done(launch_block_quantize(x, row_stride, dtype == MOE_BF16, rows, cols, q, scale, (hipStream_t)stream));
}

moe_status moe_block_pack(const void *w, int dtype, int64_t row_stride, int32_t n, int32_t k, uint8_t *q,
                          float *scale, void *stream) {
  if ((!float_type(dtype) && dtype != MOE_FP8) || n <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
  if (n > kMostBlocked || k > kMostBlocked || blocks_of(n) * blocks_of(k) > max_groups(128)) return MOE_ERR_UNSUPPORTED;
  if (!w || !al(w, dtype == MOE_F32 ? 4 : dtype == MOE_BF16 ? 2 : 1) || !q || !al(q, 16)) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_FP8 && (!scale || !al(scale, 4))) return MOE_ERR_INVALID_ARG;
  const int src = dtype == MOE_FP8 ? FMT_FP8 : dtype == MOE_BF16 ? FMT_BF16 : FMT_F32;
  return done(launch_block_pack(w, row_stride, src, n, k, q, scale, (hipStream_t)stream));
}

size_t moe_block_linear_workspace_bytes(int32_t rows, int32_t n, int32_t k, int32_t codes) {
  if (!blocked(rows) || !blocked(n) || !blocked(k)) return 0;
  LinearArgs a = {};
  a.rows = rows;
  a.n = n;
  a.k = k;
  const bool own = codes || linear_fuses(a);       // no codes are written
  return linear_part_bytes(a) + (own ? 0 : moe_block_packed_bytes(rows, k) + scale_bytes(rows, k));
}

moe_status moe_block_linear(const uint8_t *wq, const float *w_scale, int32_t n, int32_t k, const void *x,
                            int x_dtype, int64_t x_stride, const uint8_t *xq, const float *xq_scale,
                            int32_t rows, void *out, int out_dtype, void *ws, size_t ws_bytes, void *stream) {
  if (rows < 0 || n <= 0 || k <= 0 || !float_type(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (!xq != !xq_scale || (!xq && !float_type(x_dtype))) return MOE_ERR_INVALID_ARG;
  if (rows > kMostBlocked || n > kMostBlocked || k > kMostBlocked) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!wq || !al(wq, 16) || !w_scale || !al(w_scale, 4) || !out || !al(out, 16) || !al(xq, 16) || !al(xq_scale, 16) ||
      !al(ws, 16))
    return MOE_ERR_INVALID_ARG;
  if (!xq && (!x || !al(x, x_dtype == MOE_F32 ? 4 : 2))) return MOE_ERR_INVALID_ARG;
  LinearArgs a = {xq, xq_scale, wq, w_scale, out, rows, n, k, nullptr, 1};
  if (!linear_fits(a)) return MOE_ERR_UNSUPPORTED;
  const size_t need = moe_block_linear_workspace_bytes(rows, n, k, xq != nullptr);
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  a.splits = linear_splits(a);
  a.part = (float *)ws;
  if (!xq && linear_fuses(a))
    return done(launch_linear_fused(a, x, x_stride, x_dtype == MOE_BF16, out_dtype == MOE_F32, (hipStream_t)stream));
  if (!xq) {
    uint8_t *q = (uint8_t *)ws + linear_part_bytes(a);
    float *scale = (float *)(q + moe_block_packed_bytes(rows, k));
    const hipError_t err =
        launch_block_quantize(x, x_stride, x_dtype == MOE_BF16, rows, k, q, scale, (hipStream_t)stream);
    if (err != hipSuccess) return MOE_ERR_DEVICE;
    a.q = q;
    a.q_scale = scale;
  }
  return done(launch_linear(a, out_dtype == MOE_F32, (hipStream_t)stream));
}

moe_status moe_token_logprobs(const void *logits, int dtype, int64_t row_stride, const void *tokens,
                              int32_t token_bytes, int32_t rows, int32_t vocab, int32_t top, float *logprob,
                              float *entropy, float *top_logprob, int32_t *top_token, void *stream) {
  if (!logprob_args(dtype, rows, vocab, top) || (token_bytes != 4 && token_bytes != 8)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!logits || !al(logits, dtype == MOE_F32 ? 4 : 2) || !tokens || !al(tokens, token_bytes)) return MOE_ERR_INVALID_ARG;
  if (!logprob || !al(logprob, 4) || !entropy || !al(entropy, 4)) return MOE_ERR_INVALID_ARG;
  if (top && (!top_logprob || !al(top_logprob, 4) || !top_token || !al(top_token, 4))) return MOE_ERR_INVALID_ARG;
  const LogprobArgs a = {logits, row_stride, tokens, dtype == MOE_BF16, token_bytes, rows, vocab, top,
                         logprob, entropy, top_logprob, top_token};
  return done(launch_logprobs(a, (hipStream_t)stream));
}

}  // extern "C"
