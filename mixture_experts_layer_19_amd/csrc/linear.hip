// linear.hip -- matrix product in E4M3 with fp32 scales: one per row and 128 columns
// of the activations, one per 128 x 128 of the weights.
//
//   y[r, n] = sum_b s_x[r, b] s_w[n / 128, b] sum_{k in block b} q_x[r, k] q_w[n, k]
//
// Codes of both sides lie in blocks of 16 rows x 128 columns, 2 KiB, [rows / 16][cols / 128],
// in the order the 16x16x128 instruction takes them: [half][lane][16 bytes], lane l with
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

// Sums over one block of 128 columns.  The 8-bit instruction adds a lane's products by
// eights, aligned to the largest of the eight and cut off 13 bits below its power of
// two (measured; the sums of eights are then added in fp32).  On products of one block
// that is 5e-5 of the result at worst, against half a step of 2e-3 where the result is
// rounded to bf16.  Where it is not, the codes go to bf16, which holds them exactly, and
// through instructions of half the rate that add in fp32.
template <bool F32>
__device__ __forceinline__ f32x4 block_product(const i32x4 &w0, const i32x4 &w1, const i32x4 &x0, const i32x4 &x1) {
  f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (!F32) {
    const i32x8 w = __builtin_shufflevector(w0, w1, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 x = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, y, 0, 0, 0, 0, 0, 0);      // no scales
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    auto bf16 = [&](const i32x4 &c) MOE_INLINE {
      const uint2 a = e4m3_to_bf16x4((uint32_t)c[2 * (i & 1)], 127), b = e4m3_to_bf16x4((uint32_t)c[2 * (i & 1) + 1], 127);
      return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
    };
    y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16(i < 2 ? w0 : w1), bf16(i < 2 ? x0 : x1), y, 0, 0, 0);
  }
  return y;
}

// ----------------------------------------------------------------------------- codes

// Scale of a block with the largest magnitude am: am times the fp32 number 1/448, rounded
// to fp32, 0 for zeros, at least the smallest normal number otherwise; NaN for an infinity
// or NaN.
__device__ __forceinline__ float block_scale(float am) {
  return am > 0.0f && am < INFINITY ? fmaxf(am * (1.0f / 448.0f), 0x1p-126f) : am == 0.0f ? 0.0f : __builtin_nanf("");
}
// E4M3 code of v / scale: the quotient in 64 bits (a multiplication by the inverse and a
// correction, which makes quotients that 64 bits hold exact), then to the code by way of
// fp32 rounded to odd, so that what lies next to the border of two codes falls on its side.
struct Quotient {
  double scale, inv;
  __device__ __forceinline__ Quotient(float s) : scale(s), inv(s == 0.0f ? 0.0 : 1.0 / (double)s) {}
  __device__ __forceinline__ float operator()(float v) const {
    const double q = (double)v * inv;
    return round_f32<true>(fma(fma(-q, scale, (double)v), inv, q));
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
// n of 16 consecutive elements of a row, the rest 0
template <bool BF16, bool VEC>
__device__ __forceinline__ void load16(const void *p, long long i, int n, float (&v)[16]) {
  if (VEC && n >= 16) {
    float a[8], b[8];
    load8<BF16>(p, i, a);
    load8<BF16>(p, i + 8, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = a[j], v[8 + j] = b[j];
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

// Activations: a wave takes 8 rows of one block, 8 lanes a row, 16 elements a lane.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void block_quantize_kernel(const void *x, long long stride, int rows, int cols,
                                                             uint8_t *q, float *scale, int first) {
  const int blocks = (cols + kBlk - 1) / kBlk, rows16 = (rows + 15) / 16 * 16;
  const long long unit = ((long long)blockIdx.x * 4 + (threadIdx.x >> 6));
  const int lane = threadIdx.x & 63, b = (int)(unit % blocks), i = lane & 7;
  const long long row = first + unit / blocks * 8 + (lane >> 3);
  if (row >= rows16) return;
  const int k = b * kBlk + 16 * i;
  float v[16];
  load16<BF16, VEC>(x, row * stride + k, row < rows ? min(cols - k, 16) : 0, v);
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
                                                         float *scale, int first) {
  __shared__ float red[2];
  const int blocks = (cols + kBlk - 1) / kBlk, tid = threadIdx.x;
  const long long unit = (long long)first + blockIdx.x;
  const int b = (int)(unit % blocks), i = tid & 7, k = b * kBlk + 16 * i, n16 = (n + 15) / 16 * 16;
  const long long row0 = unit / blocks * kBlk;
  float am = 0.0f, v[16];
  if constexpr (!CODES) {
    for (long long row = row0 + (tid >> 3); row < row0 + kBlk && row < n; row += 16) {
      load16<BF16, false>(w, row * stride + k, min(cols - k, 16), v);
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
      load16<BF16, false>(w, row * stride + k, have, v);
      *(i32x4 *)to = codes16(v, quot);
    }
  }
  if (!CODES && tid == 0) scale[unit] = s;
}

// ----------------------------------------------------------------------------- products

// Four neighbouring columns n .. n + 3 of row r (those below a.n).
template <bool F32>
__device__ __forceinline__ void store4(const LinearArgs &a, long long r, int n, const f32x4 &y) {
  const long long at = r * a.n + n;
  if (a.n % 4 == 0) {
    if (n >= a.n) return;
    if constexpr (F32) *(f32x4 *)((float *)a.out + at) = y;
    else *(uint2 *)((uint16_t *)a.out + at) = make_uint2(bf16_pack2(y[0], y[1]), bf16_pack2(y[2], y[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.n) {
        if constexpr (F32) ((float *)a.out)[at + i] = y[i];
        else ((uint16_t *)a.out)[at + i] = (uint16_t)bf16_pack2(y[i], 0.0f);
      }
  }
}

// Few rows: 16 RT rows and 16 columns a workgroup, its four waves a quarter of the
// blocks each, their sums added in the waves' order.
template <bool F32, int RT>
__global__ __launch_bounds__(256) void block_rows_kernel(LinearArgs a) {
  __shared__ f32x4 part[4][RT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = (a.k + kBlk - 1) / kBlk, rows16 = (a.rows + 15) / 16 * 16;
  const int nb = blockIdx.x;
  const int b0 = (int)((long long)blocks * wave / 4), b1 = (int)((long long)blocks * (wave + 1) / 4);
  const uint8_t *w = a.w + (long long)nb * blocks * kBlkBytes + lane * 16;
  const float *ws = a.w_scale + (long long)(nb / 8) * blocks;
  f32x4 acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    const i32x4 w0 = *(const i32x4 *)(w + (long long)b * kBlkBytes);
    const i32x4 w1 = *(const i32x4 *)(w + (long long)b * kBlkBytes + 1024);
    const float sw = ws[b];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int rb = min(t, rows16 / 16 - 1);
      const uint8_t *x = a.q + ((long long)rb * blocks + b) * kBlkBytes + lane * 16;
      const f32x4 p = block_product<F32>(w0, w1, *(const i32x4 *)x, *(const i32x4 *)(x + 1024));
      const float s = a.q_scale[(long long)b * rows16 + rb * 16 + (lane & 15)] * sw;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(p[i], s, acc[t][i]);
    }
  }
#pragma unroll
  for (int t = 0; t < RT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < RT; t += 4) {
    const f32x4 y = ((part[0][t][lane] + part[1][t][lane]) + part[2][t][lane]) + part[3][t][lane];
    const long long r = (long long)t * 16 + (lane & 15);
    if (r < a.rows) store4<F32>(a, r, nb * 16 + 4 * (lane >> 4), y);
  }
}

// Many rows: a tile of TM rows x TN columns a workgroup, WM x WN of it a wave.  Both
// sides' blocks of 128 columns go from memory to the LDS without passing registers, as
// they lie (a wave's read of a fragment is 1 KiB in a row), the next one's while this
// one's products run.
template <int TM, int TN, int WM, int WN>
struct TileCfg {
  static constexpr int waves_n = TN / WN, waves = TM / WM * waves_n, threads = 64 * waves;
  static constexpr int x_blocks = TM / 16, w_blocks = TN / 16, blocks = x_blocks + w_blocks;
  static constexpr int stage = blocks * kBlkBytes + TM * 4;      // and the rows' scales
  static constexpr int lds = 2 * stage;
  static_assert(blocks % waves == 0 && TM % 64 == 0);
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

template <bool F32, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(64 * (TM / WM) * (TN / WN), 2) void block_tile_kernel(LinearArgs a, int tiles_m, int tiles_n) {
  using C = TileCfg<TM, TN, WM, WN>;
  constexpr int MT = WM / 16, NT = WN / 16, PER = C::blocks / C::waves, GROUP = 4;
  extern __shared__ __align__(16) uint8_t lds[];
  const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t *)lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::waves_n, wn = wave % C::waves_n;
  const int blocks = (a.k + kBlk - 1) / kBlk, x16 = (a.rows + 15) / 16, n16 = (a.n + 15) / 16;

  // Workgroups go round the eight XCDs; each takes a run of tiles, GROUP row tiles by
  // all column tiles at a time, so that those that run together share its L2.
  const int total = tiles_m * tiles_n, per = (total + 7) / 8, tile = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (tile >= total) return;
  const int first = tile / (GROUP * tiles_n) * GROUP, group = min(GROUP, tiles_m - first), in = tile - first * tiles_n;
  const int tm = first + in % group, tn = in / group;

  // this wave's blocks of a stage, rows of the tile before columns
  const uint8_t *src[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int blk = wave * PER + i;
    src[i] = blk < C::x_blocks ? a.q + (long long)min(tm * C::x_blocks + blk, x16 - 1) * blocks * kBlkBytes
                               : a.w + (long long)min(tn * C::w_blocks + blk - C::x_blocks, n16 - 1) * blocks * kBlkBytes;
  }
  const float *row_scale = a.q_scale + tm * TM;
  const uint32_t s_off = (min(tm * TM + wave * 64 + lane, x16 * 16 - 1) - tm * TM) * 4;
  const float *col_scale = a.w_scale + (long long)min((tn * TN + wn * WN) / 128, (n16 - 1) / 8) * blocks;
  auto load = [&](int b) MOE_INLINE {
    const uint32_t to = lds0 + (b & 1) * C::stage;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      block_to_lds(to + (wave * PER + i) * kBlkBytes, src[i] + (long long)b * kBlkBytes, lane * 16);
    if (wave < TM / 64)
      word_to_lds(to + C::blocks * kBlkBytes + wave * 256, row_scale + (long long)b * x16 * 16, s_off);
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[t][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  load(0);
  float sw = col_scale[0];
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  asm volatile("" : "+v"(sw));
  for (int b = 0; b < blocks; ++b) {
    float sw_next = sw;
    if (b + 1 < blocks) {
      sw_next = col_scale[b + 1];
      load(b + 1);
    }
    const uint8_t *st = lds + (b & 1) * C::stage + lane * 16;
    const float *sc = (const float *)(lds + (b & 1) * C::stage + C::blocks * kBlkBytes) + wm * WM + (lane & 15);
    i32x4 w0[NT], w1[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint8_t *p = st + (C::x_blocks + wn * NT + j) * kBlkBytes;
      w0[j] = *(const i32x4 *)p;
      w1[j] = *(const i32x4 *)(p + 1024);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint8_t *p = st + (wm * MT + t) * kBlkBytes;
      const i32x4 x0 = *(const i32x4 *)p, x1 = *(const i32x4 *)(p + 1024);
      const float s = sc[16 * t] * sw;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x4 y = block_product<F32>(w0[j], w1[j], x0, x1);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(y[i], s, acc[t][j][i]);
      }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    asm volatile("" : "+v"(sw_next));
    sw = sw_next;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const long long r = (long long)tm * TM + wm * WM + t * 16 + (lane & 15);
    if (r < a.rows)
#pragma unroll
      for (int j = 0; j < NT; ++j) store4<F32>(a, r, tn * TN + wn * WN + j * 16 + 4 * (lane >> 4), acc[t][j]);
  }
}

// ----------------------------------------------------------------------------- launches

namespace {
template <bool F32, int TM, int TN, int WM, int WN>
hipError_t tiles(const LinearArgs &a, hipStream_t s) {
  using C = TileCfg<TM, TN, WM, WN>;
  static OncePerDevice once;
  const auto kernel = block_tile_kernel<F32, TM, TN, WM, WN>;
  const hipError_t err = allow_lds(once, (const void *)kernel, C::lds);
  if (err != hipSuccess) return err;
  const int tm = (a.rows + TM - 1) / TM, tn = (a.n + TN - 1) / TN;
  kernel<<<(unsigned)(((long long)tm * tn + 7) / 8 * 8), C::threads, C::lds, s>>>(a, tm, tn);
  return hipGetLastError();
}

template <bool F32>
hipError_t linear(const LinearArgs &a, hipStream_t s) {
  const int n16 = (a.n + 15) / 16, rb = (a.rows + 15) / 16;
  if (a.rows > 64) {
    const long long big = ((a.rows + 255ll) / 256) * ((a.n + 255ll) / 256);
    return big >= 256 ? tiles<F32, 256, 256, 128, 64>(a, s) : tiles<F32, 128, 128, 64, 64>(a, s);
  }
  if (rb <= 1) block_rows_kernel<F32, 1><<<n16, 256, 0, s>>>(a);
  else if (rb <= 2) block_rows_kernel<F32, 2><<<n16, 256, 0, s>>>(a);
  else block_rows_kernel<F32, 4><<<n16, 256, 0, s>>>(a);
  return hipGetLastError();
}
}  // namespace

bool linear_fits(int rows, int n) {
  const long long n16 = (n + 15ll) / 16, tiles = ((rows + 127ll) / 128) * ((n + 127ll) / 128);
  return rows <= 64 ? n16 <= max_groups(256) : tiles + 8 <= max_groups(512);
}

hipError_t launch_block_quantize(const void *x, long long stride, int is_bf16, int rows, int cols, uint8_t *q,
                                 float *scale, hipStream_t s) {
  const int blocks = (int)((cols + (kBlk - 1ll)) / kBlk);
  const long long rows16 = (rows + 15ll) / 16 * 16, e = is_bf16 ? 8 : 4;
  const bool vec = ((uintptr_t)x & 15) == 0 && (rows == 1 || stride % e == 0);
  // rows of a launch: a multiple of 8
  long long most = max_groups(256) * 4 / blocks * 8;
  if (most == 0) return hipErrorInvalidValue;
  for (long long row0 = 0; row0 < rows16; row0 += most) {
    const long long n = rows16 - row0 < most ? rows16 - row0 : most;
    const unsigned grid = (unsigned)((n / 8 * blocks + 3) / 4);
    if (is_bf16 && vec) block_quantize_kernel<true, true><<<grid, 256, 0, s>>>(x, stride, rows, cols, q, scale, (int)row0);
    else if (is_bf16) block_quantize_kernel<true, false><<<grid, 256, 0, s>>>(x, stride, rows, cols, q, scale, (int)row0);
    else if (vec) block_quantize_kernel<false, true><<<grid, 256, 0, s>>>(x, stride, rows, cols, q, scale, (int)row0);
    else block_quantize_kernel<false, false><<<grid, 256, 0, s>>>(x, stride, rows, cols, q, scale, (int)row0);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_block_pack(const void *w, long long stride, int src, int n, int cols, uint8_t *q, float *scale,
                             hipStream_t s) {
  const long long units = ((n + (kBlk - 1ll)) / kBlk) * ((cols + (kBlk - 1ll)) / kBlk);
  const unsigned grid = (unsigned)units;
  if (src == FMT_FP8) block_pack_kernel<false, true><<<grid, 128, 0, s>>>(w, stride, n, cols, q, scale, 0);
  else if (src == FMT_BF16) block_pack_kernel<true, false><<<grid, 128, 0, s>>>(w, stride, n, cols, q, scale, 0);
  else block_pack_kernel<false, false><<<grid, 128, 0, s>>>(w, stride, n, cols, q, scale, 0);
  return hipGetLastError();
}

hipError_t launch_linear(const LinearArgs &a, int f32_out, hipStream_t s) {
  return f32_out ? linear<true>(a, s) : linear<false>(a, s);
}

}  // namespace moe
