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

}  // extern "C"
