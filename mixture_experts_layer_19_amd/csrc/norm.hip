// norm.hip -- RMS norm with the residual's addition and an output in 8 bits.
//
//   s = x + residual                      (fp32)
//   y = s / sqrt(mean(s^2) + eps) * weight
//   residual_out = round(s), y_out = round(y)
//   q = E4M3 codes of y: under one E8M0 scale per 32 (MX) or of y / fp8_scale
//
// The sum is held in fp32 (exact for nearly all bf16 operands), the statistic,
// y and y / fp8_scale in 64 bits, and every output is rounded once from them: y
// goes to bf16 and to the codes by way of fp32 rounded to odd, which keeps what
// lies below and above a tie or a power of two apart (y in fp32 moved the scale,
// and with it 32 codes, of a block whose maximum lay next to a power of two).  The
// 64-bit instructions cost 1.5% (8192 x 4096 bf16 with MX codes: 55.0 -> 55.8 us);
// the rest of them runs under the loads.
//
// Bound by memory: a bf16 row with MX output moves 9.03 bytes an element
// (8192 x 4096: 60 us, 5.0 TB/s; a copy reaches 4.9).
// One pass: a row stays in registers between the sum of squares and its use,
// in one wave up to 2048 elements (no LDS, no barrier) and in a workgroup of
// 256 up to 8192; longer rows, rows that are not 16-byte aligned and odd
// lengths are read a second time (norm_loop_kernel: 2048 x 16384 bf16 with MX codes
// 90 us, 3.4 TB/s; 8192 x 4095, element by element, 236 us, 1.3 TB/s).
#include "block_common.hpp"

namespace moe {

template <bool BF16>
__device__ __forceinline__ void load8(const void *p, long long i, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 u = *(const uint4 *)((const uint16_t *)p + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
    const float4 a = *(const float4 *)((const float *)p + i);
    const float4 b = *(const float4 *)((const float *)p + i + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void *p, long long i, const float (&v)[8]) {
  if constexpr (BF16) {
    *(uint4 *)((uint16_t *)p + i) = make_uint4(bf16_pack2(v[0], v[1]), bf16_pack2(v[2], v[3]),
                                               bf16_pack2(v[4], v[5]), bf16_pack2(v[6], v[7]));
  } else {
    *(float4 *)((float *)p + i) = make_float4(v[0], v[1], v[2], v[3]);
    *(float4 *)((float *)p + i + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}
// n of 8 elements, one at a time
template <bool BF16>
__device__ __forceinline__ void load_n(const void *p, long long i, int n, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.0f;
    if (j < n) {
      if constexpr (BF16) v[j] = bf16_to_f32(((const uint16_t *)p)[i + j]);
      else v[j] = ((const float *)p)[i + j];
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void store_n(void *p, long long i, int n, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) {
      if constexpr (BF16) ((uint16_t *)p)[i + j] = (uint16_t)bf16_pack2(v[j], 0.0f);
      else ((float *)p)[i + j] = v[j];
    }
}

// d rounded to fp32: to nearest, or to odd (towards zero, then the last bit set if
// anything was cut off), from which one more rounding to fewer bits is as if from d.
template <bool ODD>
__device__ __forceinline__ float round_f32(double d) {
  const float n = (float)d;
  if constexpr (!ODD) return n;
  uint32_t u = __float_as_uint(n);
  u -= fabs((double)n) > fabs(d) ? 1u : 0u;
  return __uint_as_float(u | ((double)n != d ? 1u : 0u));
}
// y of 8 elements: `out` to be stored as the row's type, `code` for the codes (FP8:
// y by the scale, in 64 bits as y is; the scale's inverse, 8192 x 4096 57.5 us,
// adds a rounding of 2^-53 to the quotient's, 67.8).
template <bool BF16, int Q>
__device__ __forceinline__ void norm8(const NormArgs &a, const float (&v)[8], double rs, const float (&w)[8],
                                      float (&out)[8], float (&code)[8]) {
  const double rq = Q == FMT_FP8 ? 1.0 / (double)a.fp8_scale : 1.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const double d = (double)v[j] * rs * (double)w[j];
    const float odd = round_f32<true>(d);
    code[j] = Q == FMT_FP8 ? round_f32<true>(d * rq) : odd;
    out[j] = BF16 ? odd : round_f32<false>(d);
  }
}

// 8-bit output of 8 consecutive elements (n of them present; MX: all, four
// neighbouring lanes hold one block of 32 and take its maximum together).
template <int Q>
__device__ __forceinline__ void store_codes(const NormArgs &a, long long i, int n, bool whole,
                                            const float (&y)[8]) {
  if constexpr (Q == FMT_MX8) {
    float am = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(y[j]));
    am = fmaxf(am, __shfl_xor(am, 1, 64));
    am = fmaxf(am, __shfl_xor(am, 2, 64));
    const uint32_t sb = mx_scale_byte(am);
    const float inv = mx_inv_scale(sb);
    const uint2 w = make_uint2(e4m3_pack4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                               e4m3_pack4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
    if (n > 0) {
      *(uint2 *)(a.q + i) = w;
      if ((threadIdx.x & 3) == 0) a.q_scale[i >> 5] = (uint8_t)sb;
    }
  } else if constexpr (Q == FMT_FP8) {
    const uint2 w = make_uint2(e4m3_pack4(y[0], y[1], y[2], y[3]), e4m3_pack4(y[4], y[5], y[6], y[7]));
    if (whole) {
      *(uint2 *)(a.q + i) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) a.q[i + j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
    }
  }
}

// Sum over LANES threads: a wave, or a workgroup of 256.
template <int LANES>
__device__ __forceinline__ double row_sum(double v, double *red) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0] + red[1] + red[2] + red[3];
  }
  return v;
}

// A row per LANES threads, NV runs of 8 elements a thread, in registers.
template <bool BF16, int Q, int LANES, int NV>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  __shared__ double red[4];
  const int lane = threadIdx.x % LANES;
  const int row = blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (LANES <= 64 && row >= a.rows) return;
  const int nvec = a.hidden / 8;
  float v[NV][8];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + i * LANES;
    if (c < nvec) {
      load8<BF16>(a.x, row * a.x_stride + 8 * c, v[i]);
      if (a.residual) {
        float r[8];
        load8<BF16>(a.residual, row * a.residual_stride + 8 * c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += r[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fma((double)v[i][j], (double)v[i][j], ss);
  }
  const double rs = 1.0 / sqrt(row_sum<LANES>(ss, red) / a.hidden + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = lane + i * LANES;
    const bool in = c < nvec;
    const long long at = (long long)row * a.hidden + 8 * c;
    float y[8], code[8];
    if (in) {
      if (a.residual_out) store8<BF16>(a.residual_out, at, v[i]);
      float w[8];
      load8<BF16>(a.weight, 8 * c, w);
      norm8<BF16, Q>(a, v[i], rs, w, y, code);
      if (a.y) store8<BF16>(a.y, at, y);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) code[j] = 0.0f;
    }
    store_codes<Q>(a, at, in ? 8 : 0, in, code);
  }
}

// Any length and alignment: a workgroup per row, the row read twice.
// Everything is written in the second pass, so outputs may be the inputs.
template <bool BF16, int Q, bool VEC>
__global__ __launch_bounds__(256) void norm_loop_kernel(NormArgs a) {
  __shared__ double red[4];
  const int row = blockIdx.x, tid = threadIdx.x;
  const int nvec = a.hidden / 8 + (a.hidden % 8 != 0);
  auto load = [&](int c, float (&v)[8]) {
    const int n = min(8, a.hidden - 8 * c);
    float r[8];
    if constexpr (VEC) load8<BF16>(a.x, row * a.x_stride + 8 * c, v);
    else load_n<BF16>(a.x, row * a.x_stride + 8 * c, n, v);
    if (a.residual) {
      if constexpr (VEC) load8<BF16>(a.residual, row * a.residual_stride + 8 * c, r);
      else load_n<BF16>(a.residual, row * a.residual_stride + 8 * c, n, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
    return n;
  };
  double ss = 0.0;
  for (int c = tid; c < nvec; c += 256) {
    float v[8];
    load(c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fma((double)v[j], (double)v[j], ss);
  }
  const double rs = 1.0 / sqrt(row_sum<256>(ss, red) / a.hidden + a.eps);
  for (int c0 = 0; c0 < nvec; c0 += 256) {       // every lane takes part in the block maxima
    const int c = c0 + tid;
    const long long at = (long long)row * a.hidden + 8 * c;
    float y[8], code[8];
    int n = 0;
    if (c < nvec) {
      float v[8], w[8];
      n = load(c, v);
      if constexpr (VEC) {
        load8<BF16>(a.weight, 8 * c, w);
        if (a.residual_out) store8<BF16>(a.residual_out, at, v);
      } else {
        load_n<BF16>(a.weight, 8 * c, n, w);
        if (a.residual_out) store_n<BF16>(a.residual_out, at, n, v);
      }
      norm8<BF16, Q>(a, v, rs, w, y, code);
      if (a.y) {
        if constexpr (VEC) store8<BF16>(a.y, at, y);
        else store_n<BF16>(a.y, at, n, y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) code[j] = 0.0f;
    }
    store_codes<Q>(a, at, n, VEC && n > 0, code);
  }
}

namespace {
bool al16(const void *p) { return ((uintptr_t)p & 15) == 0; }

template <bool BF16, int Q>
void launch(const NormArgs &a, hipStream_t s) {
  const long long e = BF16 ? 8 : 4;              // elements of 16 bytes
  const bool vec = a.hidden % 8 == 0 && a.x_stride % e == 0 && a.residual_stride % e == 0 &&
                   al16(a.x) && al16(a.residual) && al16(a.weight) && al16(a.residual_out) &&
                   al16(a.y);
  const int nvec = a.hidden / 8;
  const dim3 g1((a.rows + 3) / 4), g4(a.rows);
  if (!vec) norm_loop_kernel<BF16, Q, false><<<g4, 256, 0, s>>>(a);
  else if (nvec <= 64) norm_kernel<BF16, Q, 64, 1><<<g1, 256, 0, s>>>(a);
  else if (nvec <= 128) norm_kernel<BF16, Q, 64, 2><<<g1, 256, 0, s>>>(a);
  else if (nvec <= 256) norm_kernel<BF16, Q, 64, 4><<<g1, 256, 0, s>>>(a);
  else if (nvec <= 512) norm_kernel<BF16, Q, 256, 2><<<g4, 256, 0, s>>>(a);
  else if (nvec <= 1024) norm_kernel<BF16, Q, 256, 4><<<g4, 256, 0, s>>>(a);
  else norm_loop_kernel<BF16, Q, true><<<g4, 256, 0, s>>>(a);
}
}  // namespace

hipError_t launch_rms_norm(const NormArgs &all, int is_bf16, int q_fmt, hipStream_t s) {
  constexpr int kRows = 1 << 23;                 // of a launch: up to a workgroup each
  static_assert(kRows <= max_groups(256), "rows of a launch");
  const int e = is_bf16 ? 2 : 4;
  for (long long r0 = 0; r0 < all.rows; r0 += kRows) {
    NormArgs a = all;
    auto skip = [&](auto *&p, long long bytes) {
      if (p) p = (std::remove_reference_t<decltype(p)>)((const uint8_t *)p + r0 * bytes);
    };
    skip(a.x, all.x_stride * e);
    skip(a.residual, all.residual_stride * e);
    skip(a.residual_out, (long long)all.hidden * e);
    skip(a.y, (long long)all.hidden * e);
    skip(a.q, all.hidden);
    skip(a.q_scale, all.hidden / 32);
    a.rows = (int)(all.rows - r0 < kRows ? all.rows - r0 : kRows);
    if (is_bf16) {
      if (q_fmt == FMT_MX8) launch<true, FMT_MX8>(a, s);
      else if (q_fmt == FMT_FP8) launch<true, FMT_FP8>(a, s);
      else launch<true, -1>(a, s);
    } else {
      if (q_fmt == FMT_MX8) launch<false, FMT_MX8>(a, s);
      else if (q_fmt == FMT_FP8) launch<false, FMT_FP8>(a, s);
      else launch<false, -1>(a, s);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
