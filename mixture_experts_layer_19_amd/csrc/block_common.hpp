// block_common.hpp -- device helpers shared by the norm, cache and attention
// kernels.
#pragma once
#include "block_launch.hpp"
#include "moe_common.hpp"

namespace moe {

typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(2))) int i32x2;

constexpr float kNegBig = -3.402823466e38f;   // running maximum before any key: finite, below every score
// The weight of a score s is exp2(s * scale - reference).  As one fused operation
// that does not round the product as the reference was rounded, which scales all
// weights of a row alike, by up to 2^(|reference| / 2^24): 2^16 at 2^28, but past
// fp32 from 2^31 on.  So the product is rounded first (x s - r in two steps): where
// memory is the bound, always; where the vector units are, only in half tiles with a
// score whose exponent (frexp) is above far_exponent, a product of 2^27 or more.
// There (chunks of 640-1408 tokens) the test costs 0.6% (861 -> 866 us), one of the
// scaled maximum 2%, products rounded everywhere 5%.
__device__ __forceinline__ float mul_sub(float x, float s, float r) {
#pragma clang fp contract(off)
  return x * s - r;
}
__device__ __forceinline__ int far_exponent(float scale) { return 28 + 126 - (int)(__float_as_uint(scale) >> 23); }

// v, its magnitude limited to 448; a NaN stays one.
__device__ __forceinline__ float e4m3_clamp(float v) {
  return fabsf(v) > 448.0f ? copysignf(448.0f, v) : v;
}
// E4M3 codes of four values, round to nearest even, saturating, NaN kept (the
// conversion instruction itself turns values above 464 into NaN).
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(a), e4m3_clamp(b), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(c), e4m3_clamp(d), w, true);
  return (uint32_t)w;
}
// Two bf16 (packed) of two fp32 values, round to nearest even, NaN kept.
__device__ __forceinline__ uint32_t bf16_pack2(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
// Four bf16 of four E4M3 codes times the power of two with E8M0 byte `sb`.
// The instruction takes the exponent field of its scale operand, so byte 0 is
// 2^-127 and byte 255 NaN; every product is exact in bf16.
__device__ __forceinline__ uint2 e4m3_to_bf16x4(uint32_t codes, uint32_t sb) {
  const float s = __uint_as_float(sb << 23);
  return make_uint2(
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, s, false)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, s, true)));
}

// Largest / sum over the two half waves and over the four rows of 16 lanes.
__device__ __forceinline__ float max_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float max_rows16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max_half(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_rows16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return sum_half(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Inclusive sums over the lanes of a wave: within rows of 16, then the rows'
// last lanes carried into the rows behind them.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast 15 to rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast 31 to rows 2 and 3
  return v;
}

// ----------------------------------------------------------------------------- batch geometry

// One sequence of a batch.  Whatever the device arrays hold, rows stay inside
// [0, rows) and keys inside the table's capacity.
struct SeqGeo {
  int r0, n;       // first row and number of new rows
  int pos0;        // position of the first new token (negative: before the sequence)
  int len;         // tokens that the table can hold of kv_len
};
__device__ __forceinline__ SeqGeo seq_geo(const KvArgs &c, int s) {
  SeqGeo g;
  const int o0 = c.offsets[s], o1 = c.offsets[s + 1], kvl = max(c.kv_len[s], 0);
  g.r0 = min(max(o0, 0), c.rows);
  g.n = min(max(o1, g.r0), c.rows) - g.r0;
  g.pos0 = kvl - g.n;
  g.n = min(g.n, c.max_rows);      // the launch holds no more
  const long long cap = (long long)c.max_pages << c.page_shift;
  g.len = (int)min((long long)kvl, cap);
  return g;
}

// The same in scalar registers (all lanes hold the same).
__device__ __forceinline__ SeqGeo uniform(SeqGeo g) {
  g.r0 = __builtin_amdgcn_readfirstlane(g.r0);
  g.n = __builtin_amdgcn_readfirstlane(g.n);
  g.pos0 = __builtin_amdgcn_readfirstlane(g.pos0);
  g.len = __builtin_amdgcn_readfirstlane(g.len);
  return g;
}

// Sequence of row r (every lane of the wave asks for the same r): the last
// one that starts at or before it; -1 where no sequence holds the row.  g: its
// geometry, from the same loads.
__device__ __forceinline__ int seq_of_row(const KvArgs &c, int r, SeqGeo &g) {
  const int lane = threadIdx.x & 63;
  int found = -1;
  for (int s0 = 0; s0 < c.seqs; s0 += 64) {
    const int s = min(s0 + lane, c.seqs - 1);
    const SeqGeo own = seq_geo(c, s);
    const unsigned long long m = __ballot(s0 + lane < c.seqs && c.offsets[s] <= r);
    if (!m) break;
    const int l = 63 - __clzll((long long)m);
    found = s0 + l;
    g.r0 = __builtin_amdgcn_readlane(own.r0, l);
    g.n = __builtin_amdgcn_readlane(own.n, l);
    g.pos0 = __builtin_amdgcn_readlane(own.pos0, l);
    g.len = __builtin_amdgcn_readlane(own.len, l);
    if (m != ~0ull) break;
  }
  return found;
}

// Index of a key's row in the pool, (page * kv_heads + head) * page_size +
// slot, or kNoRow where the table holds no page for it.  (A pool has fewer
// than 2^32 - 1 rows.)
constexpr uint32_t kNoRow = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t pool_row(const KvArgs &c, int page, int head, int key) {
  const uint32_t row = (((uint32_t)page * (uint32_t)c.kv_heads + (uint32_t)head) << c.page_shift) |
                       ((uint32_t)key & ((1u << c.page_shift) - 1u));
  return (unsigned)page < (unsigned)c.num_pages ? row : kNoRow;
}

}  // namespace moe
