// rotate.hip -- RMS norm of each head of the queries and keys, their rotation by
// position, and in the same pass, where asked for, the write of keys and values into
// the paged cache.
//
//   n = x / sqrt(mean(x^2) + eps) * weight           over one head
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t), t = position * inv_freq[i]
//
// over the pairs (i, i + rotary / 2), or the neighbours (2i, 2i + 1), of the first
// `rotary` elements.  With the weight and the turn of a row folded into two factors an
// element, y_j = (x_j c_j + x_partner s_j) / rms.
//
// The mean of squares is fp32, and where it nears the ends of fp32's range taken again in
// 64 bits, with x multiplied by a power of two near 1 / rms; the angle is held in 64
// bits, reduced to a quarter turn before its sine and cosine are taken (their Taylor
// series, whose first terms left out are below 2^-52) and rounded to fp32.  The rest is
// fp32, for keys that go into codes 64 bits, and every output is rounded once from it.
//
// Bound by memory: a bf16 element is 4 bytes in and out (8925 rows of 64 + 2 x 8 heads of
// 128 into MX-fp8 78 us, 4.5 TB/s; 2311 of 32 + 4 fp32 heads 17.0 us, 5.0 TB/s).  A wave holds 64 pieces of 8
// elements, 512 / head_dim heads of one row, so that a lane's place in its head, and with
// it the factors, stay what they are; four such steps are loaded at once.
#include "block_common.hpp"

namespace moe {

enum RotateTo { TO_ROWS, TO_POOL, TO_MX };     // keys to k_out; keys and values to the cache

// sin (x) and cos (y) of a 64-bit angle.
__device__ __forceinline__ double2 sin_cos(double angle) {
  const double n = rint(angle * 0.63661977236758134308);         // quarter turns
  double r = fma(-n, 1.57079632679489655800, angle);             // pi / 2 in two parts
  r = fma(-n, 6.12323399573676603587e-17, r);
  const double z = r * r;
  double s = -1.0 / 1307674368000.0, c = 1.0 / 20922789888000.0;  // 1 / 15!, 1 / 16!
  s = fma(s, z, 1.0 / 6227020800.0);
  s = fma(s, z, -1.0 / 39916800.0);
  s = fma(s, z, 1.0 / 362880.0);
  s = fma(s, z, -1.0 / 5040.0);
  s = fma(s, z, 1.0 / 120.0);
  s = fma(s, z, -1.0 / 6.0);
  s = fma(s * z, r, r);
  c = fma(c, z, -1.0 / 87178291200.0);
  c = fma(c, z, 1.0 / 479001600.0);
  c = fma(c, z, -1.0 / 3628800.0);
  c = fma(c, z, 1.0 / 40320.0);
  c = fma(c, z, -1.0 / 720.0);
  c = fma(c, z, 1.0 / 24.0);
  c = fma(c, z, -0.5);
  c = fma(c, z, 1.0);
  // which quarter: n mod 4 (n is whole and below 2^52; a larger angle, or none, gives NaN)
  const double quarter = fabs(n) < 4503599627370496.0 ? n - 4.0 * rint(n * 0.25) : __builtin_nan("");
  if (!(quarter == quarter)) return make_double2(quarter, quarter);
  const int q = (int)quarter & 3;
  const double sn = q & 1 ? c : s, cs = q & 1 ? s : c;
  return make_double2(q & 2 ? -sn : sn, (q + 1) & 2 ? -cs : cs);
}

// A row of L lanes a head of 8 L elements; `parts` waves share a row's heads.
// (Five waves a SIMD: at four, which the steps in 64 bits would take, 8925 rows 90.5 us.)
template <bool BF16, int TO, int L>
__global__ __launch_bounds__(256, 5) void rotate_kernel(RotateArgs a, int parts, int first) {
  constexpr int HEADS = 64 / L, HD = 8 * L;
  const int lane = threadIdx.x & 63, piece = lane % L, d0 = 8 * piece;
  const uint32_t unit = blockIdx.x * 4u + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t in_launch = unit / (uint32_t)parts;
  const int part = (int)(unit - in_launch * (uint32_t)parts);
  if (in_launch >= (uint32_t)(a.c.rows - first)) return;
  const int row = first + (int)in_launch;

  int pos;
  uint32_t place = kNoRow;
  bool found = true;
  if constexpr (TO == TO_ROWS) {
    pos = a.positions[row];
  } else {
    SeqGeo g = {};
    const int s = seq_of_row(a.c, row, g);
    pos = g.pos0 + (row - g.r0);
    found = s >= 0 && row - g.r0 < g.n && pos >= 0 && pos < g.len;
    if (found) place = pool_row(a.c, a.c.table[(long long)s * a.c.max_pages + (pos >> a.c.page_shift)], 0, pos);
  }

  // The row's turn: lane i takes pairs i and i + 64, and each lane fetches those of
  // its eight elements.
  const int half = a.rotary / 2;
  const double2 t0 = sin_cos((double)pos * a.inv_freq[min(lane, half - 1)]);
  const double2 t1 = half > 64 ? sin_cos((double)pos * a.inv_freq[min(lane + 64, half - 1)]) : t0;
  // of element d: sine (with the partner's sign) and cosine, as T
  auto turn_of = [&](int d, auto &sine, auto &cosine) MOE_INLINE {
    using T = std::remove_reference_t<decltype(sine)>;
    const int i = a.interleaved ? d >> 1 : d < half ? d : d - half;
    T s = __shfl((T)t0.x, i & 63, 64), c = __shfl((T)t0.y, i & 63, 64);
    if (half > 64) {
      const T s1 = __shfl((T)t1.x, i & 63, 64), c1 = __shfl((T)t1.y, i & 63, 64);
      s = i & 64 ? s1 : s;
      c = i & 64 ? c1 : c;
    }
    const bool minus = a.interleaved ? !(d & 1) : d < half;
    cosine = d < a.rotary ? c : (T)1;
    sine = d < a.rotary ? (minus ? -s : s) : (T)0;
  };
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) turn_of(d0 + j, sn[j], cs[j]);
  // the lane that holds the partners (this one: neighbours, and elements not turned)
  const int hop = a.interleaved || d0 >= a.rotary ? 0 : d0 < half ? half / 8 : -half / 8;
  const int partner = lane + hop;

  const int q_steps = (a.heads + HEADS - 1) / HEADS, k_steps = (a.c.kv_heads + HEADS - 1) / HEADS;
  const int steps = q_steps + (TO == TO_ROWS ? k_steps : 2 * k_steps);
  const int begin = (int)((long long)steps * part / parts), end = (int)((long long)steps * (part + 1) / parts);

  float cw[8], sw[8];                            // the factors: weight and turn
  auto weights = [&](const void *w) MOE_INLINE {
    float own[8], other[8];
    load8<BF16>(w, d0, own);
    load8<BF16>(w, d0 + 8 * hop, other);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // (the neighbour of an element that is not turned is not used: sn is 0)
      const float o = a.after ? own[j] : a.interleaved ? own[j ^ 1] : other[j];
      cw[j] = own[j] * cs[j];
      sw[j] = o * sn[j];
    }
  };

  double kc[8], ks[8];                           // those of keys that go into codes
  auto weights_64 = [&]() MOE_INLINE {
    float own[8], other[8];
    load8<BF16>(a.k_weight, d0, own);
    load8<BF16>(a.k_weight, d0 + 8 * hop, other);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      turn_of(d0 + j, ks[j], kc[j]);
      kc[j] *= own[j];
      ks[j] *= a.after ? own[j] : a.interleaved ? own[j ^ 1] : other[j];
    }
  };

  // steps [s0, s1) of one of q, k, v; KIND 0, 1, 2
  auto run = [&](auto kind, int s0, int s1, const void *src, long long row_stride, long long head_stride,
                 int heads) MOE_INLINE {
    constexpr int KIND = decltype(kind)::value, BATCH = KIND == 1 && TO == TO_MX ? 2 : 4;
    for (int sb = s0; sb < s1; sb += BATCH) {
      float v[BATCH][8];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int h = min(min(sb + b, s1 - 1) * HEADS + lane / L, heads - 1);
        load8<BF16>(src, (long long)row * row_stride + h * head_stride + d0, v[b]);
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        if (sb + b >= s1) break;
        const int h = (sb + b) * HEADS + lane / L;
        float y[8];
        if constexpr (KIND == 1 && TO == TO_MX) {
          // What goes into codes: in 64 bits, and to the codes by way of fp32 rounded to
          // odd, so that a value next to the border of two, or a block's largest next to a
          // power of two, falls on its side (8925 rows, 8 of 80 heads: 80.7 -> 84.1 us).
          double ss = 0.0;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fma((double)v[b][j], (double)v[b][j], ss);
#pragma unroll
          for (int m = 1; m < L; m <<= 1) ss += __shfl_xor(ss, m, 64);
          const double ms = ss * (1.0 / HD) + a.eps, r0 = __builtin_amdgcn_rsq(ms), t = fma(-ms * r0, r0, 1.0);
          const double r = fabs(t) < 1.0 ? fma(r0 * t, fma(0.375, t, 0.5), r0) : r0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = a.interleaved && d0 + j < a.rotary ? v[b][j ^ 1] : __shfl(v[b][j], partner, 64);
            y[j] = round_f32<true>(fma((double)v[b][j], kc[j], (double)x * ks[j]) * r);
          }
        } else if constexpr (KIND < 2) {
          float fs = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) fs = fmaf(v[b][j], v[b][j], fs);
#pragma unroll
          for (int m = 1; m < L; m <<= 1) fs += __shfl_xor(fs, m, 64);
          float ms = fmaf(fs, 1.0f / HD, a.eps);
          int e = 0;
          // squares that overflow, or are so small that some are lost: in 64 bits, with x
          // multiplied by a power of two near 1 / rms first
          if (__ballot(!(ms > 0x1p-80f && ms < 0x1p80f))) {
            double ss = 0.0;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fma((double)v[b][j], (double)v[b][j], ss);
#pragma unroll
            for (int m = 1; m < L; m <<= 1) ss += __shfl_xor(ss, m, 64);
            ss = ss * (1.0 / HD) + a.eps;
            e = __builtin_amdgcn_frexp_exp(ss) >> 1;
            ms = (float)ldexp(ss, -2 * e);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[b][j] = ldexpf(v[b][j], -e);
          }
          const float r0 = __builtin_amdgcn_rsqf(ms), t = fmaf(-ms * r0, r0, 1.0f);
          const float r = fabsf(t) < 1.0f ? fmaf(0.5f * r0, t, r0) : r0;     // (0, infinity and NaN as they are)
          if (a.interleaved) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              y[j] = fmaf(v[b][j], cw[j], d0 + j < a.rotary ? v[b][j ^ 1] * sw[j] : 0.0f) * r;
          } else {                               // (what is not turned is its own partner, times 0)
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = fmaf(v[b][j], cw[j], __shfl(v[b][j], partner, 64) * sw[j]) * r;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = v[b][j];
        }
        if (h >= heads) continue;
        if constexpr (KIND == 0 || TO == TO_ROWS) {
          if (!found) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = 0.0f;
          }
          store8<BF16>(KIND == 0 ? a.q_out : a.k_out, ((long long)row * heads + h) * HD + d0, y);
        } else {
          if (place == kNoRow) continue;
          const long long dst = (long long)(place + ((uint32_t)h << a.c.page_shift)) * HD + d0;
          uint8_t *pool = KIND == 1 ? a.c.k : a.c.v;
          if constexpr (TO == TO_POOL) {
            store8<BF16>(pool, dst, y);
          } else {
            float am = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(y[j]));
            am = fmaxf(am, __shfl_xor(am, 1, 64));       // four lanes hold a block of 32
            am = fmaxf(am, __shfl_xor(am, 2, 64));
            const uint32_t sb8 = mx_scale_byte(am);
            const float inv = mx_inv_scale(sb8);
            *(uint2 *)(pool + dst) =
                make_uint2(e4m3_pack4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                           e4m3_pack4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
            if ((lane & 3) == 0) (KIND == 1 ? a.c.k_scale : a.c.v_scale)[dst >> 5] = (uint8_t)sb8;
          }
        }
      }
    }
  };
  const int q_end = min(end, q_steps), k_end = min(end, q_steps + k_steps);
  if (begin < q_end) {
    weights(a.q_weight);
    run(std::integral_constant<int, 0>{}, begin, q_end, a.q, a.q_row, a.q_head, a.heads);
  }
  if (TO != TO_ROWS && place == kNoRow) return;
  if (max(begin, q_steps) < k_end) {
    if constexpr (TO == TO_MX) weights_64();
    else weights(a.k_weight);
    run(std::integral_constant<int, 1>{}, max(begin - q_steps, 0), k_end - q_steps, a.k, a.k_row, a.k_head,
        a.c.kv_heads);
  }
  if constexpr (TO != TO_ROWS)
    if (k_end < end)
      run(std::integral_constant<int, 2>{}, max(begin - q_steps - k_steps, 0), end - q_steps - k_steps, a.v, a.v_row,
          a.v_head, a.c.kv_heads);
}

namespace {
template <bool BF16, int TO, int L>
hipError_t launch(const RotateArgs &a, hipStream_t s) {
  constexpr int HEADS = 64 / L;
  const int k_steps = (a.c.kv_heads + HEADS - 1) / HEADS;
  const int steps = (a.heads + HEADS - 1) / HEADS + (TO == TO_ROWS ? 1 : 2) * k_steps;
  // Steps of a wave: 4 as long as its waves are few (64 rows of 64 + 2 x 8 heads of 128
  // into MX-fp8 6.0 us, with 10 steps 9.2), else 10, which find their row's place and
  // turn half as often (8925 rows: 89.8 and 80.7 us; 8192 without a cache 72.7 and 60.6).
  const int of_wave = (long long)a.c.rows * ((steps + 3) / 4) < 16384 ? 4 : 10;
  const int parts = (steps + of_wave - 1) / of_wave;
  const long long most = max_groups(256) * 4 / parts;     // rows of a launch
  for (long long row0 = 0; row0 < a.c.rows; row0 += most) {
    const long long rows = a.c.rows - row0 < most ? a.c.rows - row0 : most;
    rotate_kernel<BF16, TO, L><<<(unsigned)((rows * parts + 3) / 4), 256, 0, s>>>(a, parts, (int)row0);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}
template <bool BF16, int TO>
hipError_t launch_dim(const RotateArgs &a, hipStream_t s) {
  return a.c.head_dim == 64 ? launch<BF16, TO, 8>(a, s)
         : a.c.head_dim == 128 ? launch<BF16, TO, 16>(a, s) : launch<BF16, TO, 32>(a, s);
}
}  // namespace

hipError_t launch_rotate(const RotateArgs &a, int is_bf16, int into_cache, hipStream_t s) {
  if (!into_cache) return is_bf16 ? launch_dim<true, TO_ROWS>(a, s) : launch_dim<false, TO_ROWS>(a, s);
  return a.c.fmt == FMT_F32 ? launch_dim<false, TO_POOL>(a, s)
         : a.c.fmt == FMT_BF16 ? launch_dim<true, TO_POOL>(a, s) : launch_dim<true, TO_MX>(a, s);
}

}  // namespace moe
