// attn_common.hpp -- what the attention kernels share: which keys a query row
// sees, the order in which key tiles are visited, loads of keys and queries.
//
//   out[r, h] = sum_j softmax_j(scale * q[r, h] . k[j, h / group]) v[j, h / group]
//
// over the keys j <= pos(r) of the row's sequence; with a window W also
// j > pos(r) - W or j < sinks.  A row that sees no key gives zeros.  Scores,
// maxima, sums and the output accumulate in fp32; the softmax runs on powers
// of two (scale * log2(e) is folded into the scores).
//
// With a bf16 or MX cache the weights are rounded to bf16 for the second product,
// whose matrix instructions take bf16 (fp32 ones run at a tenth of the rate); their
// sum is taken before that, in fp32.  Half a step of bf16 a key, independent from key
// to key: the results lie 0.0023 of their size from 64 bits, 0.0017 with fp32
// weights, of which the output's own rounding to bf16 is nearly all.
//
// The rows of one sequence and KV head are the pairs (token, query head of
// the group), token-major: row m is token m / group, head m % group.  So the
// query heads that share keys fill a matrix tile together.
#pragma once
#include "block_common.hpp"
#include "once_per_device.hpp"

namespace moe {

// Allow `bytes` of dynamic LDS to a kernel on the current device; `once`: of that kernel.
inline hipError_t allow_lds(OncePerDevice &once, const void *kernel, int bytes) {
  int device = 0;
  const hipError_t err = hipGetDevice(&device);
  if (err != hipSuccess) return err;
  return (hipError_t)once(device, [&] {
    return (int)hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

// Key tiles of BK keys that tokens [i0, i1] of a sequence visit: the tiles
// that hold sinks, then those of the window.
template <int BK>
struct KeyRange {
  int sink_tiles, first, tiles;
  __device__ __forceinline__ KeyRange(const SeqGeo &g, int i0, int i1, int window, int sinks) {
    const int hi = min(max(g.pos0 + i1 + 1, 0), g.len);
    const int lo = window ? min(max(g.pos0 + i0 - window + 1, 0), hi) : 0;
    first = lo / BK;
    sink_tiles = window ? min((min(sinks, hi) + BK - 1) / BK, first) : 0;
    tiles = sink_tiles + (hi + BK - 1) / BK - first;
  }
  __device__ __forceinline__ int key(int t) const {   // first key of the t-th tile
    return (t < sink_tiles ? t : first + t - sink_tiles) * BK;
  }
};

// Keys that one query row sees: [lo, hi) and [0, sinks).
struct RowMask {
  int lo, hi, sinks;
  __device__ __forceinline__ RowMask(const SeqGeo &g, int token, bool in, int window, int nsinks) {
    const int pos = g.pos0 + token;
    hi = in ? min(pos + 1, g.len) : 0;
    lo = window ? pos - window + 1 : 0;
    sinks = nsinks;
  }
  __device__ __forceinline__ bool sees(int key) const { return key < hi && (key >= lo || key < sinks); }
};

// Values that are not finite.  The second product multiplies every key of a
// tile, also with the zero weights of rows that do not see it; so in tiles of
// which some row does not see every key, elements that are not finite are zero in
// LDS and are added afterwards, by add_not_finite, to the rows that do see them.
//
// Whether a 32-bit word of a pool holds one (MX: a NaN code).
template <int F>
__device__ __forceinline__ bool word_not_finite(uint32_t w) {
  if constexpr (F == FMT_MX8) return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  else if constexpr (F == FMT_BF16) return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
  else return (w & 0x7F800000u) == 0x7F800000u;
}
// E8M0 byte from which an E4M3 value may be infinite in bf16 (255: is NaN)
constexpr uint32_t kScaleOverflow = 247;
// A word of LDS (two bf16, or one fp32) with zeros in their place.
template <int F>
__device__ __forceinline__ uint32_t word_finite(uint32_t w) {
  if constexpr (F == FMT_F32) return (w & 0x7F800000u) == 0x7F800000u ? 0u : w;
  const uint32_t lo = (w & 0x7F80u) == 0x7F80u ? 0u : w & 0xFFFFu;
  return lo | ((w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u);
}
// What is not finite of elements [d, d + 4) of pool row r, zero elsewhere.
template <int F, int HD>
__device__ __forceinline__ f32x4 not_finite4(const KvArgs &c, uint32_t r, int d) {
  const long long at = (long long)r * HD + d;
  f32x4 v;
  if constexpr (F == FMT_F32) {
    v = *(const f32x4 *)(c.v + 4 * at);
  } else {
    uint2 w;
    if constexpr (F == FMT_BF16) w = *(const uint2 *)(c.v + 2 * at);
    else w = e4m3_to_bf16x4(*(const uint32_t *)(c.v + at), c.v_scale[at >> 5]);
    v = f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
              __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)};
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = word_not_finite<FMT_F32>(__float_as_uint(v[i])) ? v[i] : 0.0f;
  return v;
}

// Zeros for the rows before the first and past the last sequence.
template <int F, int HD>
__device__ __forceinline__ void clear_free_rows(const AttnArgs &a) {
  const KvArgs &c = a.c;
  const int first = min(max(c.offsets[0], 0), c.rows), last = min(max(c.offsets[c.seqs], 0), c.rows);
  if (first == 0 && last == c.rows) return;
  const long long per_row = (long long)a.heads * HD * (F == FMT_F32 ? 4 : 2) / 16;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < c.rows * per_row;
       i += (long long)gridDim.x * blockDim.x) {
    const long long r = i / per_row;
    if (r < first || r >= last) ((uint4 *)a.out)[i] = make_uint4(0, 0, 0, 0);
  }
}

}  // namespace moe
