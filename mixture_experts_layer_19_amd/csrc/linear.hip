// linear.hip -- matrix product in E4M3 with fp32 scales: one per row and 128 columns
// of the activations, one per 128 x 128 of the weights.
//
//   y[r, n] = sum_b s_x[r, b] s_w[n / 128, b] sum_{k in block b} q_x[r, k] q_w[n, k]
//
// Codes of both sides lie in blocks of 16 rows x 128 columns, 2 KiB, [rows / 16][cols / 128],
// so that a lane's share is two reads of 16 bytes: [half][lane][16 bytes], lane l with
// row l % 16 and columns 32 (l / 16) + 16 half of the block.  (Which columns a lane
// holds does not matter to a product as long as both sides agree.)  Rows and columns are
// filled up with zeros.  Activation scales are [cols / 128][rows], rows filled up to 16.
//
// Weights are the instruction's first operand, so a lane's four sums belong to one row
// of the activations and four neighbouring columns of the result, and one factor
// s_x s_w serves all four: a block's product starts from zero and is added with it.
#include "block_common.hpp"

namespace moe {

constexpr int kBlk = 128;                        // columns of a block
constexpr int kBlkBytes = 16 * kBlk;             // 16 rows of it
constexpr int kFused = 8192;                     // codes that every workgroup makes itself, at most

// Sums over one block of 128 columns, in fp32: the codes go to bf16, which holds them
// exactly, and through instructions that add in fp32.  The 8-bit instruction has twice the
// rate (8192 x 4096 by 10240: 290 us, these 495), but adds a lane's products by eights,
// aligned to the largest of the eight and cut off 13 bits below its power of two
// (measured): up to 7 x 2^-13 of that largest product, always towards zero, and where large
// products cancel, all of what is left.
__device__ __forceinline__ f32x4 block_product(const i32x8 &w, const i32x8 &x) {
  f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    auto bf16 = [&](const i32x8 &c) MOE_INLINE {
      const uint2 a = e4m3_to_bf16x4((uint32_t)c[2 * i], 127), b = e4m3_to_bf16x4((uint32_t)c[2 * i + 1], 127);
      return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
    };
    y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16(w), bf16(x), y, 0, 0, 0);
  }
  return y;
}
// A lane's 32 bytes of a block at p (its own 16 of the first half)
__device__ __forceinline__ i32x8 fragment(const uint8_t *p) {
  return __builtin_shufflevector(*(const i32x4 *)p, *(const i32x4 *)(p + 1024), 0, 1, 2, 3, 4, 5, 6, 7);
}

// ----------------------------------------------------------------------------- codes

// Scale of a block with the largest magnitude am: am times the fp32 number 1/448, rounded
// to fp32, 0 for zeros, at least the smallest normal number otherwise; NaN for an infinity
// or NaN.  Not am / 448, which differs by a step for some am: this is what torch on the GPU
// makes of a division by the constant 448, so that activations quantised with it have the
// same scales and codes.
__device__ __forceinline__ float block_scale(float am) {
  return am > 0.0f && am < INFINITY ? fmaxf(am * (1.0f / 448.0f), 0x1p-126f) : am == 0.0f ? 0.0f : __builtin_nanf("");
}
// v / scale rounded to odd (towards zero, then the last bit set if anything was cut
// off), from which the code, of 4 bits, is as if from the exact quotient: what lies next
// to the border of two codes falls on its side.  A quotient within a step of the exact one,
// and the sign of what is left, which a fused operation holds exactly: scales near the
// lower end of fp32 are taken up from it with their values, and of values below
// scale / 2^11, where it might be lost, the code is 0 anyway.  (In 64 bits, with three
// conversions a value at a quarter of the rate: 8192 x 4096 27.3 us.)
struct Quotient {
  float up, scale, inv;
  __device__ __forceinline__ Quotient(float s) : up(s < 0x1p-70f ? 0x1p64f : 1.0f), scale(s * up),
                                                 inv(s == 0.0f ? 0.0f : 1.0f / scale) {}
  __device__ __forceinline__ float operator()(float v) const {
    const float x = v * up, q0 = x * inv, q = fmaf(fmaf(-q0, scale, x), inv, q0), rest = fmaf(-q, scale, x);
    const uint32_t b = __float_as_uint(q), below = (__float_as_uint(rest) ^ b) >> 31;   // the quotient is: one step down
    return __uint_as_float(rest != 0.0f ? (b - below) | 1u : b);
  }
};
// 16 codes of 16 consecutive values
__device__ __forceinline__ i32x4 codes16(const float (&v)[16], const Quotient &q) {
  i32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    r[j] = (int)e4m3_pack4(q(v[4 * j]), q(v[4 * j + 1]), q(v[4 * j + 2]), q(v[4 * j + 3]));
  return r;
}
// n of 16 consecutive elements of a row, the rest 0.  (Vector loads need only an element's
// alignment; a row that starts between two 16-byte borders takes some lines twice.)
typedef i32x4 __attribute__((aligned(2))) i32x4_at2;
typedef i32x4 __attribute__((aligned(4))) i32x4_at4;
template <bool BF16>
__device__ __forceinline__ void load16(const void *p, long long i, int n, float (&v)[16]) {
  if (n >= 16) {
    if constexpr (BF16) {
      const i32x4_at2 *at = (const i32x4_at2 *)((const uint16_t *)p + i);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t w = (uint32_t)at[j / 8][j / 2 % 4];
        v[j] = __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
      }
    } else {
      const i32x4_at4 *at = (const i32x4_at4 *)((const float *)p + i);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __int_as_float(at[j / 4][j % 4]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      v[j] = 0.0f;
      if (j < n) {
        if constexpr (BF16) v[j] = bf16_to_f32(((const uint16_t *)p)[i + j]);
        else v[j] = ((const float *)p)[i + j];
      }
    }
  }
}
__device__ __forceinline__ float largest16(const float (&v)[16]) {
  float am = 0.0f;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    am = fmaxf(am, fabsf(v[j]));
    nan |= v[j] != v[j];
  }
  return nan ? INFINITY : am;                    // either makes the scale NaN
}

// Activations: a wave takes 8 rows of one block, 8 lanes a row, 16 elements a lane
// (8192 x 4096 bf16: 20.4 us, 4.9 TB/s).
template <bool BF16>
__global__ __launch_bounds__(256) void block_quantize_kernel(const void *x, long long stride, int rows, int cols,
                                                             uint8_t *q, float *scale, int first) {
  const int blocks = (cols + kBlk - 1) / kBlk, rows16 = (rows + 15) / 16 * 16;
  const uint32_t unit = blockIdx.x * 4u + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t of_rows = unit / (uint32_t)blocks;
  const int lane = threadIdx.x & 63, b = (int)(unit - of_rows * (uint32_t)blocks), i = lane & 7;
  const long long row = first + (long long)of_rows * 8 + (lane >> 3);
  if (row >= rows16) return;
  const int k = b * kBlk + 16 * i;
  float v[16];
  load16<BF16>(x, row * stride + k, row < rows ? min(cols - k, 16) : 0, v);
  float am = largest16(v);
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) am = fmaxf(am, __shfl_xor(am, m, 64));
  const float s = block_scale(am);
  // columns 32 (i / 2) + 16 (i % 2): half i % 2 of lane group i / 2
  uint8_t *to = q + (row / 16 * blocks + b) * kBlkBytes + (i & 1) * 1024 + ((i >> 1) * 16 + row % 16) * 16;
  *(i32x4 *)to = codes16(v, Quotient(s));
  if (i == 0) scale[(long long)b * rows16 + row] = s;
}

// Weights: a workgroup takes 128 x 128, 128 threads 8 lanes a row, 16 rows at a time.
// CODES: they are codes already and only change places.
template <bool BF16, bool CODES>
__global__ __launch_bounds__(128) void block_pack_kernel(const void *w, long long stride, int n, int cols, uint8_t *q,
                                                         float *scale) {
  __shared__ float red[2];
  const int blocks = (cols + kBlk - 1) / kBlk, tid = threadIdx.x;
  const long long unit = blockIdx.x;
  const int b = (int)(unit % blocks), i = tid & 7, k = b * kBlk + 16 * i, n16 = (n + 15) / 16 * 16;
  const long long row0 = unit / blocks * kBlk;
  float am = 0.0f, v[16];
  if constexpr (!CODES) {
    for (long long row = row0 + (tid >> 3); row < row0 + kBlk && row < n; row += 16) {
      load16<BF16>(w, row * stride + k, min(cols - k, 16), v);
      am = fmaxf(am, largest16(v));
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) am = fmaxf(am, __shfl_xor(am, m, 64));
    if ((tid & 63) == 0) red[tid >> 6] = am;
    __syncthreads();
    am = fmaxf(red[0], red[1]);
  }
  const float s = block_scale(am);
  const Quotient quot(s);
  for (long long row = row0 + (tid >> 3); row < row0 + kBlk && row < n16; row += 16) {
    uint8_t *to = q + (row / 16 * blocks + b) * kBlkBytes + (i & 1) * 1024 + ((i >> 1) * 16 + row % 16) * 16;
    const int have = row < n ? min(cols - k, 16) : 0;
    if constexpr (CODES) {
      const uint8_t *from = (const uint8_t *)w + row * stride + k;
      if (have == 16 && ((uintptr_t)from & 15) == 0) {
        *(i32x4 *)to = *(const i32x4 *)from;
      } else {
        for (int j = 0; j < 16; ++j) to[j] = j < have ? from[j] : 0;
      }
    } else {
      load16<BF16>(w, row * stride + k, have, v);
      *(i32x4 *)to = codes16(v, quot);
    }
  }
  if (!CODES && tid == 0) scale[unit] = s;
}

// ----------------------------------------------------------------------------- products

// Four neighbouring columns n .. n + 3 of row r (those below a.n), at any alignment of an
// element.
typedef uint2 __attribute__((aligned(2))) uint2_at2;
typedef f32x4 __attribute__((aligned(4))) f32x4_at4;
template <bool F32>
__device__ __forceinline__ void store4(const LinearArgs &a, long long r, int n, const f32x4 &y) {
  const long long at = r * a.n + n;
  if (n + 4 <= a.n) {
    if constexpr (F32) *(f32x4_at4 *)((float *)a.out + at) = y;
    else *(uint2_at2 *)((uint16_t *)a.out + at) = make_uint2(bf16_pack2(y[0], y[1]), bf16_pack2(y[2], y[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (n + i < a.n) {
        if constexpr (F32) ((float *)a.out)[at + i] = y[i];
        else ((uint16_t *)a.out)[at + i] = (uint16_t)bf16_pack2(y[i], 0.0f);
      }
  }
}

// Few rows: 16 RT rows and 16 CT columns a workgroup, its KW waves a share of the
// blocks each, their sums added in the waves' order.  The next block's codes are on their
// way while one's products run.  Bound by memory: the weights once from HBM (one row of
// 4096 by 120832: 86 us, 5.8 TB/s), and the activations' codes from the L2 by every
// workgroup, which with 64 rows of 4096 by 10240 columns cost 15.4 us at 16 columns each, 13.1
// at 48 (one row 9.6 and 10.6).
template <bool F32, int RT, int CT, int KW>
__global__ __launch_bounds__(64 * KW) void block_rows_kernel(LinearArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  f32x4 (*part)[RT * CT][64] = (f32x4 (*)[RT * CT][64])lds;      // [KW]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = (a.k + kBlk - 1) / kBlk, x16 = (a.rows + 15) / 16, n16 = (a.n + 15) / 16;
  const int nb = blockIdx.x * CT;
  const int b0 = (int)((long long)blocks * wave / KW), b1 = (int)((long long)blocks * (wave + 1) / KW);
  const uint8_t *w[CT], *x[RT];
  const float *ws[CT], *xs[RT];
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const int n = min(nb + j, n16 - 1);
    w[j] = a.w + (long long)n * blocks * kBlkBytes;
    ws[j] = a.w_scale + (long long)(n / 8) * blocks;
  }
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int r = min(t, x16 - 1);
    x[t] = a.q + (long long)r * blocks * kBlkBytes;
    xs[t] = a.q_scale + r * 16;
  }
  struct Block {
    i32x8 w[CT], x[RT];
    float ws[CT], xs[RT];
  };
  auto read = [&](int b, Block &o) MOE_INLINE {
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      o.w[j] = fragment(w[j] + (long long)b * kBlkBytes + lane * 16);
      o.ws[j] = ws[j][b];
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      o.x[t] = fragment(x[t] + (long long)b * kBlkBytes + lane * 16);
      o.xs[t] = xs[t][(long long)b * x16 * 16 + (lane & 15)];
    }
  };
  f32x4 acc[RT][CT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](const Block &o) MOE_INLINE {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        const f32x4 p = block_product(o.w[j], o.x[t]);
        const float s = o.xs[t] * o.ws[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(p[i], s, acc[t][j][i]);
      }
  };
  if (b0 < b1) {
    Block one, two;
    read(b0, one);
    int b = b0;
    for (; b + 2 < b1; b += 2) {
      read(b + 1, two);
      multiply(one);
      read(b + 2, one);
      multiply(two);
    }
    if (b + 1 < b1) {
      read(b + 1, two);
      multiply(one);
      multiply(two);
    } else {
      multiply(one);
    }
  }
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int j = 0; j < CT; ++j) part[wave][t * CT + j][lane] = acc[t][j];
  __syncthreads();
  for (int i = wave; i < RT * CT; i += KW) {
    f32x4 y = part[0][i][lane];
#pragma unroll
    for (int v = 1; v < KW; ++v) y += part[v][i][lane];
    const long long r = (long long)(i / CT) * 16 + (lane & 15);
    if (r < a.rows) store4<F32>(a, r, (nb + i % CT) * 16 + 4 * (lane >> 4), y);
  }
}

// LDS of the codes and scales of block_fused_kernel.
__host__ __device__ __forceinline__ int fused_codes_bytes(int rows, int k) {
  const int blocks = (k + kBlk - 1) / kBlk;
  return (rows * (blocks * (kBlk + 4) + 16) + 15) / 16 * 16;
}

// The least work: block_rows_kernel with CT = 1 whose workgroups each make the codes of
// all activations themselves, in the LDS, in place of a launch before it.  Sums are in the
// same order.  (One row of 8192 by 4096: 10.2 us, in two launches 11.5.)
template <bool F32, bool BF16, int RT, int KW>
__global__ __launch_bounds__(64 * KW) void block_fused_kernel(LinearArgs a, const void *x, long long stride) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = (a.k + kBlk - 1) / kBlk, pitch = blocks * kBlk + 16;      // (16: banks)
  uint8_t *codes = lds;                                                        // [rows][pitch]
  float *scales = (float *)(codes + a.rows * pitch);                           // [rows][blocks]
  f32x4 (*part)[RT][64] = (f32x4 (*)[RT][64])lds;                              // [KW], when the codes are read
  const int b0 = (int)((long long)blocks * wave / KW), b1 = (int)((long long)blocks * (wave + 1) / KW);
  const uint8_t *w = a.w + (long long)blockIdx.x * blocks * kBlkBytes + lane * 16;
  const float *ws = a.w_scale + (long long)(blockIdx.x / 8) * blocks;
  constexpr int AHEAD = 4;                       // blocks of weights on their way, from here on
  i32x8 wf[AHEAD] = {};
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (b0 < b1) wf[i] = fragment(w + (long long)min(b0 + i, b1 - 1) * kBlkBytes);

  // 16 elements a thread, 8 threads a block of a row, two of them on their way at once
  const int units = a.rows * blocks * 8;
  for (int u0 = threadIdx.x; u0 < units; u0 += 2 * 64 * KW) {
    float v[2][16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int u = u0 + h * 64 * KW, row = u / 8 / blocks, k = (u / 8 - row * blocks) * kBlk + 16 * (u & 7);
      load16<BF16>(x, row * stride + k, u < units ? min(a.k - k, 16) : 0, v[h]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int u = u0 + h * 64 * KW, row = u / 8 / blocks, b = u / 8 - row * blocks;
      if (u >= units) break;
      float am = largest16(v[h]);
#pragma unroll
      for (int m = 1; m < 8; m <<= 1) am = fmaxf(am, __shfl_xor(am, m, 64));
      const float s = block_scale(am);
      *(i32x4 *)(codes + row * pitch + b * kBlk + 16 * (u & 7)) = codes16(v[h], Quotient(s));
      if ((u & 7) == 0) scales[row * blocks + b] = s;
    }
  }
  __syncthreads();

  f32x4 acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int b4 = b0; b4 < b1; b4 += AHEAD) {
#pragma unroll
    for (int h = 0; h < AHEAD; ++h) {
      const int b = b4 + h;
      if (b >= b1) break;
      const float sw = ws[b];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int row = min(16 * t + (lane & 15), a.rows - 1);
        const i32x4 *at = (const i32x4 *)(codes + row * pitch + b * kBlk + 32 * (lane >> 4));
        const i32x8 xf = __builtin_shufflevector(at[0], at[1], 0, 1, 2, 3, 4, 5, 6, 7);
        const f32x4 p = block_product(wf[h], xf);
        const float s = scales[row * blocks + b] * sw;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(p[i], s, acc[t][i]);
      }
      wf[h] = fragment(w + (long long)min(b + AHEAD, b1 - 1) * kBlkBytes);
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < RT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < RT; t += KW) {
    f32x4 y = part[0][t][lane];
#pragma unroll
    for (int v = 1; v < KW; ++v) y += part[v][t][lane];
    const long long r = (long long)t * 16 + (lane & 15);
    if (r < a.rows) store4<F32>(a, r, blockIdx.x * 16 + 4 * (lane >> 4), y);
  }
}

// Many rows: a tile of TM rows x TN columns a workgroup, WM x WN of it a wave.  Both
// sides' blocks of 128 columns go from memory to the LDS without passing registers, as
// they lie (a wave's read of a fragment is 1 KiB in a row), the next one's while this
// one's products run.  256 square of 8192 x 4096 by 10240, random codes: 495 us, 1.39 PFLOP/s
// (a large bf16 product of the library: 1.50).  Bound by the matrix units and by power:
// with codes of zeros it takes 435 us.
template <int TM, int TN, int WM, int WN>
struct TileCfg {
  static constexpr int waves_n = TN / WN, waves = TM / WM * waves_n, threads = 64 * waves;
  static constexpr int x_blocks = TM / 16, w_blocks = TN / 16, blocks = x_blocks + w_blocks;
  static constexpr int scales = (TM + 63) / 64;                  // of 64 rows
  static constexpr int stage = blocks * kBlkBytes + scales * 256;
  static constexpr int lds = 2 * stage;
  static_assert(WM % 32 == 0, "fragments take turns");
};

// 16 bytes a lane from base + offset to the LDS at `to` + 16 lane, and the same 1 KiB on.
__device__ __forceinline__ void block_to_lds(uint32_t to, const uint8_t *base, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\t"
               "global_load_lds_dwordx4 %1, %2\n\t"
               "global_load_lds_dwordx4 %1, %2 offset:1024" ::"s"(to), "v"(offset), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void word_to_lds(uint32_t to, const void *base, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory", "m0");
}

// SPLIT: a.splits workgroups share a tile's blocks and leave fp32 sums (F32) in a.part.
template <bool F32, int TM, int TN, int WM, int WN, bool SPLIT>
__global__ __launch_bounds__(64 * (TM / WM) * (TN / WN), 2) void block_tile_kernel(LinearArgs a, int tiles_m, int tiles_n) {
  using C = TileCfg<TM, TN, WM, WN>;
  constexpr int MT = WM / 16, NT = WN / 16, PER = (C::blocks + C::waves - 1) / C::waves, GROUP = 4;
  extern __shared__ __align__(16) uint8_t lds[];
  const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t *)lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::waves_n, wn = wave % C::waves_n;
  const int blocks = (a.k + kBlk - 1) / kBlk, x16 = (a.rows + 15) / 16, n16 = (a.n + 15) / 16;

  // Workgroups go round the eight XCDs; each takes a run of tiles, GROUP row tiles by
  // all column tiles at a time, so that those that run together share its L2.
  const int total = tiles_m * tiles_n, units = SPLIT ? total * a.splits : total, per = (units + 7) / 8;
  const int unit = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (unit >= units) return;
  const int split = SPLIT ? unit / total : 0, tile = unit - split * total;
  const int begin = SPLIT ? (int)((long long)blocks * split / a.splits) : 0;
  const int end = SPLIT ? (int)((long long)blocks * (split + 1) / a.splits) : blocks;
  const int first = tile / (GROUP * tiles_n) * GROUP, group = min(GROUP, tiles_m - first), in = tile - first * tiles_n;
  const int tm = first + in % group, tn = in / group;

  // this wave's blocks of a stage, rows of the tile before columns
  const uint8_t *src[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int blk = min(wave * PER + i, C::blocks - 1);          // (the last one may be loaded twice)
    src[i] = blk < C::x_blocks ? a.q + (long long)min(tm * C::x_blocks + blk, x16 - 1) * blocks * kBlkBytes
                               : a.w + (long long)min(tn * C::w_blocks + blk - C::x_blocks, n16 - 1) * blocks * kBlkBytes;
  }
  const float *row_scale = a.q_scale + tm * TM;
  const int s64 = wave % C::scales * 64;         // (more waves than that load the same ones)
  const uint32_t s_off = (min(tm * TM + s64 + lane, x16 * 16 - 1) - tm * TM) * 4;
  const float *col_scale = a.w_scale + (long long)min((tn * TN + wn * WN) / 128, (n16 - 1) / 8) * blocks;
  // part i of a stage's loads: a block, behind the last one the scales
  auto load_part = [&](int b, int i) MOE_INLINE {
    const uint32_t to = lds0 + (b & 1) * C::stage;
    if (i < PER)
      block_to_lds(to + min(wave * PER + i, C::blocks - 1) * kBlkBytes, src[i] + (long long)b * kBlkBytes, lane * 16);
    else
      word_to_lds(to + C::blocks * kBlkBytes + s64 * 4, row_scale + (long long)b * x16 * 16, s_off);
  };

  // A stage's loads: all at once as soon as its place is free, or, where the products
  // take longer than the loads, spread over the block before it, a part every row tile
  // (256 square: 504 -> 495 us; 64 square, 64 rows by 120832: 113 -> 120).
  constexpr bool SPREAD = MT >= 8;
  auto load_ahead = [&](int b) MOE_INLINE {
#pragma unroll
    for (int i = 0; i <= (SPREAD ? 0 : PER); ++i) load_part(b, i);
  };

  // Fragments are read one row tile ahead, and a tile's products are added under the
  // next one's: in this order, which the compiler's own is slower than.  Before the last
  // row tile of a block everything of it is in registers: there all waves meet, the
  // block after the next starts into its place, and the next one's first fragments are
  // read under the last tile's products.
  f32x4 acc[MT][NT], y[2][NT];
  i32x8 wf[NT], xf[2];
  float rs[2], f = 0.0f;                         // f: of the tile whose products are added
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    y[1][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  auto read_x = [&](int b, int t) MOE_INLINE {
    const uint8_t *st = lds + (b & 1) * C::stage;
    xf[t & 1] = fragment(st + (wm * MT + t) * kBlkBytes + lane * 16);
    rs[t & 1] = ((const float *)(st + C::blocks * kBlkBytes))[wm * WM + 16 * t + (lane & 15)];
  };
  auto read_w = [&](int b, int j) MOE_INLINE {
    wf[j] = fragment(lds + (b & 1) * C::stage + (C::x_blocks + wn * NT + j) * kBlkBytes + lane * 16);
  };
  auto add_up = [&](int t, int j) MOE_INLINE {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(y[t & 1][j][i], f, acc[t][j][i]);
  };

#pragma unroll
  for (int i = 0; i <= PER; ++i) load_part(begin, i);
  float sw = col_scale[begin], sw_next = sw;
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  if (end - begin > 1) {
    sw_next = col_scale[begin + 1];
    load_ahead(begin + 1);
  }
  read_x(begin, 0);
#pragma unroll
  for (int j = 0; j < NT; ++j) read_w(begin, j);
  auto block = [&](int b, auto left) MOE_INLINE {
    constexpr bool MORE = decltype(left)::value > 0;       // another block behind it, and one more
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const float own = sw;
      if (t + 1 < MT) {
        if (MORE && SPREAD) {
#pragma unroll
          for (int i = 1; i <= PER; ++i)
            if (i == t + 1 || (t + 2 == MT && i > t + 1)) load_part(b + 1, i);
        }
        read_x(b, t + 1);
      } else if constexpr (MORE) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        asm volatile("" : "+v"(sw_next));
        sw = sw_next;
        if constexpr (decltype(left)::value > 1) {
          sw_next = col_scale[b + 2];
          load_ahead(b + 2);
        }
        read_x(b + 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        y[t & 1][j] = block_product(wf[j], xf[t & 1]);
        if (MORE && t + 1 == MT) {
          __builtin_amdgcn_sched_barrier(0);
          read_w(b + 1, j);
        }
        add_up(t > 0 ? t - 1 : MT - 1, j);
        __builtin_amdgcn_sched_barrier(0);
      }
      f = rs[t & 1] * own;
      __builtin_amdgcn_sched_barrier(0);
    }
    // (or the compiler carries additions past the end of a block, in more registers
    // than there are)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        f32x4 &sum = acc[t][j];
        asm volatile("" : "+v"(sum));
      }
  };
  for (int b = begin; b + 2 < end; ++b) block(b, std::integral_constant<int, 2>{});
  if (end - begin > 1) block(end - 2, std::integral_constant<int, 1>{});
  block(end - 1, std::integral_constant<int, 0>{});
#pragma unroll
  for (int j = 0; j < NT; ++j) add_up(MT - 1, j);
  // the tile's rows out
  if constexpr (!F32) {
    // By way of the LDS, a wave's rows by themselves, so that a store is 16 bytes a lane
    // and whole lines: 16-byte pieces of a row lie turned by the row, which spreads the
    // banks.
    constexpr int PIECES = WN / 8;
    static_assert(C::waves * WM * WN * 2 <= C::lds, "the waves' rows");
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    uint8_t *own = lds + wave * WM * WN * 2;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int r = t * 16 + (lane & 15), piece = (2 * j + (lane >> 5)) ^ (r % PIECES);
        *(uint2 *)(own + (r * PIECES + piece) * 16 + (lane >> 4 & 1) * 8) =
            make_uint2(bf16_pack2(acc[t][j][0], acc[t][j][1]), bf16_pack2(acc[t][j][2], acc[t][j][3]));
      }
    const int piece = lane % PIECES, n = tn * TN + wn * WN + 8 * piece;
#pragma unroll
    for (int i = 0; i < WM * PIECES / 64; ++i) {
      const int r = i * (64 / PIECES) + lane / PIECES;
      const long long row = (long long)tm * TM + wm * WM + r;
      const i32x4 v = *(const i32x4 *)(own + (r * PIECES + (piece ^ (r % PIECES))) * 16);
      uint16_t *to = (uint16_t *)a.out + row * a.n + n;
      if (row < a.rows && n + 8 <= a.n) {
        *(i32x4_at2 *)to = v;
      } else if (row < a.rows) {
#pragma unroll
        for (int c = 0; c < 7; ++c)
          if (n + c < a.n) to[c] = (uint16_t)((uint32_t)v[c / 2] >> (16 * (c & 1)));
      }
    }
    return;
  }
  if constexpr (SPLIT) {
    a.n = (a.n + 3) / 4 * 4;
    a.out = a.part + (long long)split * a.rows * a.n;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const long long r = (long long)tm * TM + wm * WM + t * 16 + (lane & 15);
    if (r < a.rows)
#pragma unroll
      for (int j = 0; j < NT; ++j) store4<F32>(a, r, tn * TN + wn * WN + j * 16 + 4 * (lane >> 4), acc[t][j]);
  }
}

// The splits' sums together, in their order: four columns a thread.
template <bool F32>
__global__ __launch_bounds__(256) void block_join_kernel(LinearArgs a) {
  const int n4 = (a.n + 3) / 4;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x, size = (uint32_t)(a.rows * n4);      // (of at most 512 tiles)
  if (i >= size) return;
  f32x4 y = *(const f32x4 *)(a.part + 4ll * i);
  for (int s = 1; s < a.splits; ++s) y += *(const f32x4 *)(a.part + 4 * ((long long)s * size + i));
  store4<F32>(a, i / (uint32_t)n4, (int)(i % (uint32_t)n4) * 4, y);
}

// ----------------------------------------------------------------------------- launches

namespace {
template <bool F32, int TM, int TN, int WM, int WN, bool SPLIT = false>
hipError_t tiles(const LinearArgs &a, hipStream_t s) {
  using C = TileCfg<TM, TN, WM, WN>;
  static OncePerDevice once;
  const auto kernel = block_tile_kernel<F32 || SPLIT, TM, TN, WM, WN, SPLIT>;
  const hipError_t err = allow_lds(once, (const void *)kernel, C::lds);
  if (err != hipSuccess) return err;
  const int tm = (a.rows + TM - 1) / TM, tn = (a.n + TN - 1) / TN;
  kernel<<<(unsigned)(((long long)tm * tn * (SPLIT ? a.splits : 1) + 7) / 8 * 8), C::threads, C::lds, s>>>(a, tm, tn);
  if (SPLIT)
    block_join_kernel<F32><<<(unsigned)(((long long)a.rows * ((a.n + 3) / 4) + 255) / 256), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <bool F32, int RT, int CT, int KW>
hipError_t few(const LinearArgs &a, hipStream_t s) {
  constexpr int lds = KW * RT * CT * 1024;
  static OncePerDevice once;
  const hipError_t err = allow_lds(once, (const void *)block_rows_kernel<F32, RT, CT, KW>, lds);
  if (err != hipSuccess) return err;
  block_rows_kernel<F32, RT, CT, KW><<<(unsigned)((a.n + 16ll * CT - 1) / (16 * CT)), 64 * KW, lds, s>>>(a);
  return hipGetLastError();
}

// Blocks of 16 columns of a workgroup, of few rows: as many as leave the fullest of the
// 256 CUs no more of them.
int columns_of_group(int blocks) {
  int best = 1, most = 1 << 30;
  for (int ct = 1; ct <= 3; ++ct) {
    const int groups = (blocks + ct - 1) / ct, load = (groups + 255) / 256 * ct;
    if (load <= most) most = load, best = ct;
  }
  return best;
}

// Waves that share the blocks: 8 of one 16 columns, but for single rows (64 rows, 4096
// columns, k = 8192: 12.9 us, 4 waves 13.6; one row 8.4 and 8.3).
int waves_of_group(int ct, int rows) { return ct == 1 && rows > 16 ? 8 : 4; }

template <bool F32, int RT>
hipError_t few(const LinearArgs &a, hipStream_t s) {
  const int ct = columns_of_group((a.n + 15) / 16);
  if (ct == 3) return few<F32, RT, 3, 4>(a, s);
  if (ct == 2) return few<F32, RT, 2, 4>(a, s);
  return RT == 1 ? few<F32, RT, 1, 4>(a, s) : few<F32, RT, 1, 8>(a, s);
}

template <bool F32, bool BF16, int RT, int KW>
hipError_t fused(const LinearArgs &a, const void *x, long long stride, hipStream_t s) {
  const int codes = fused_codes_bytes(a.rows, a.k), lds = codes > KW * RT * 1024 ? codes : KW * RT * 1024;
  block_fused_kernel<F32, BF16, RT, KW><<<(unsigned)((a.n + 15) / 16), 64 * KW, lds, s>>>(a, x, stride);
  return hipGetLastError();
}
template <bool F32, bool BF16>
hipError_t fused(const LinearArgs &a, const void *x, long long stride, hipStream_t s) {
  if (a.rows <= 16) return fused<F32, BF16, 1, 4>(a, x, stride, s);
  const bool eight = waves_of_group(columns_of_group((a.n + 15) / 16), a.rows) == 8;
  if (a.rows <= 32) return eight ? fused<F32, BF16, 2, 8>(a, x, stride, s) : fused<F32, BF16, 2, 4>(a, x, stride, s);
  return eight ? fused<F32, BF16, 4, 8>(a, x, stride, s) : fused<F32, BF16, 4, 4>(a, x, stride, s);
}

// Which tiles: 256 or 128 square by how full their rounds are, one of the former or two of
// the latter a CU, which run at 0.87 of the speed (8192 rows, 10240 columns, k = 4096: 495
// and 567 us; 3000, 4096, 8192: 174 and 178; 2048, 4096, 8192: 170 and 120); 64 square up
// to 128 of 128 square (128, 10240, 4096: 35.1 us, 128 square 38.3; 512, 4096, 4096: 35.0 and
// 38.5; 300, 16384, 1024: 21.1 and 19.9).
long long count(const LinearArgs &a, int t) { return ((a.rows + t - 1ll) / t) * ((a.n + t - 1ll) / t); }
int tile_of(const LinearArgs &a) {
  if (a.rows <= 64) return 64;
  const long long t128 = count(a, 128), t256 = count(a, 256);
  if (t128 <= 128) return 64;
  auto full = [](long long t, long long slots) { return (double)t / (double)((t + slots - 1) / slots * slots); };
  return full(t256, 256) >= 0.87 * full(t128, 512) ? 256 : 128;
}

// (33 to 64 rows by many columns go to 64 square tiles: 64 of k = 4096 by 120832 108 us, as few
// rows 113; by 32768 36.5 and 38.3; by 10240 23.6 and 13.1.)
template <bool F32>
hipError_t linear(const LinearArgs &a, hipStream_t s) {
  if (a.rows <= 64 && (a.rows <= 32 || a.n < 32768))
    return a.rows <= 16 ? few<F32, 1>(a, s) : a.rows <= 32 ? few<F32, 2>(a, s) : few<F32, 4>(a, s);
  const int tile = tile_of(a);
  if (a.splits > 1) return tiles<F32, 64, 64, 64, 32, true>(a, s);
  return tile == 256 ? tiles<F32, 256, 256, 128, 64>(a, s)
         : tile == 128 ? tiles<F32, 128, 128, 64, 64>(a, s) : tiles<F32, 64, 64, 64, 32>(a, s);
}
}  // namespace

// Workgroups that share a tile's blocks: some 512 in all, with 8 blocks each at least
// (200 rows, 180 columns, k = 4096: 10.9 us, whole 23.3; 256, 4096, 8192: 39.6 and 44.3;
// with half the blocks each 1000, 260, 1024 takes 9.0 us, whole 8.6).
int linear_splits(const LinearArgs &a) {
  if (a.rows <= 64 || tile_of(a) != 64) return 1;
  const long long t = count(a, 64), blocks = (a.k + (kBlk - 1ll)) / kBlk;
  const long long s = 512 / t < blocks / 8 ? 512 / t : blocks / 8;
  return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}
size_t linear_part_bytes(const LinearArgs &a) {
  const int s = linear_splits(a);
  return s == 1 ? 0 : (size_t)s * a.rows * ((a.n + 3ll) / 4 * 4) * 4;
}
bool linear_fits(const LinearArgs &a) {
  // (workgroups of at most 512 threads; 64 square tiles beyond 64 rows are few)
  return (a.rows <= 64 ? (a.n + 15ll) / 16 : count(a, 128)) + 8 <= max_groups(512);
}

hipError_t launch_block_quantize(const void *x, long long stride, int is_bf16, int rows, int cols, uint8_t *q,
                                 float *scale, hipStream_t s) {
  const int blocks = (int)((cols + (kBlk - 1ll)) / kBlk);
  const long long rows16 = (rows + 15ll) / 16 * 16;
  // rows of a launch: a multiple of 8
  long long most = max_groups(256) * 4 / blocks * 8;
  if (most == 0) return hipErrorInvalidValue;
  for (long long row0 = 0; row0 < rows16; row0 += most) {
    const long long n = rows16 - row0 < most ? rows16 - row0 : most;
    const unsigned grid = (unsigned)((n / 8 * blocks + 3) / 4);
    if (is_bf16) block_quantize_kernel<true><<<grid, 256, 0, s>>>(x, stride, rows, cols, q, scale, (int)row0);
    else block_quantize_kernel<false><<<grid, 256, 0, s>>>(x, stride, rows, cols, q, scale, (int)row0);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_block_pack(const void *w, long long stride, int src, int n, int cols, uint8_t *q, float *scale,
                             hipStream_t s) {
  const long long units = ((n + (kBlk - 1ll)) / kBlk) * ((cols + (kBlk - 1ll)) / kBlk);
  const unsigned grid = (unsigned)units;
  if (src == FMT_FP8) block_pack_kernel<false, true><<<grid, 128, 0, s>>>(w, stride, n, cols, q, scale);
  else if (src == FMT_BF16) block_pack_kernel<true, false><<<grid, 128, 0, s>>>(w, stride, n, cols, q, scale);
  else block_pack_kernel<false, false><<<grid, 128, 0, s>>>(w, stride, n, cols, q, scale);
  return hipGetLastError();
}

// Activations small enough that every workgroup makes their codes, and few enough of
// those (4096 columns: one row of k = 4096 7.6 us, in two launches 9.4, and 4 us less on
// the host; of 8192 10.2 and 11.5; of 12288 14.5 and 13.8; three of 4096 9.9 and 9.3; 10240
// columns: two rows of 4096 11.6 and 14.0, three 14.2 and 13.9).  At most 10 KB of LDS, or 32 of
// sums.
bool linear_fuses(const LinearArgs &a) {
  return a.rows <= 64 && a.n <= 16384 && (long long)a.rows * ((a.k + (kBlk - 1ll)) / kBlk) * kBlk <= kFused;
}

hipError_t launch_linear_fused(const LinearArgs &a, const void *x, long long stride, int is_bf16, int f32_out,
                               hipStream_t s) {
  if (f32_out) return is_bf16 ? fused<true, true>(a, x, stride, s) : fused<true, false>(a, x, stride, s);
  return is_bf16 ? fused<false, true>(a, x, stride, s) : fused<false, false>(a, x, stride, s);
}

hipError_t launch_linear(const LinearArgs &a, int f32_out, hipStream_t s) {
  return f32_out ? linear<true>(a, s) : linear<false>(a, s);
}

}  // namespace moe
