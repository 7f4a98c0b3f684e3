// kv.hip -- the paged KV cache: new tokens written (quantised to MX-fp8 where
// the cache is) and read back.
//
// The pool holds K and V as [num_pages][kv_heads][page][head_dim]: one head's
// tokens of a page are contiguous, which is what attention over one KV head
// reads.  A row r of a batch is token kv_len[s] - offsets[s + 1] + r of its
// sequence s.  Rows of no sequence, and tokens for which the table holds no
// page, are not written and read back as zeros.
//
// Bound by memory: a bf16 token's head of 128 is 256 bytes on one side and
// 132 (MX) or 256 on the other.  A workgroup takes R rows, a thread 16 bytes of
// activations at a time, four pieces in flight; when writing, the first four
// are on their way while the rows' places are looked up.  Measured, 8 heads of
// 128: 8900 tokens written into MX-fp8 15.0 us (3.7 TB/s), bf16 13.8 (5.3), fp32
// 28.4 (5.1); 37000 tokens read from MX-fp8 48.7 us (4.6 TB/s), bf16 50.6 (5.8),
// fp32 115 (5.1).
#include "block_common.hpp"

namespace moe {

struct KvIo {
  void *k, *v;                 // rows outside the pool
  long long k_row, k_head, v_row, v_head;
  int piece_shift;             // log2 of the 16-byte pieces of a head
  uint32_t per_row;            // 2^32 / (2 kv_heads), rounded up
  int first;                   // first row of this launch
};

// Place of each of the workgroup's rows in the pool, head 0 (kNoRow: none).
template <int R>
__device__ __forceinline__ void find_rows(const KvArgs &c, int row0, uint32_t *place) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int i = 0; i < R / 4; ++i) {
    const int r = row0 + 4 * i + wave;
    uint32_t p = kNoRow;
    if (r < c.rows) {
      SeqGeo g;
      const int s = seq_of_row(c, r, g);
      if (s >= 0) {
        const int pos = g.pos0 + (r - g.r0);
        if (r - g.r0 < g.n && pos >= 0 && pos < g.len)
          p = pool_row(c, c.table[(long long)s * c.max_pages + (pos >> c.page_shift)], 0, pos);
      }
    }
    if ((threadIdx.x & 63) == 0) place[4 * i + wave] = p;
  }
}

// Piece i of a workgroup: its row, side (0 K, 1 V), head and first element.
// (No divisions: they would cost more than the rest of the kernel.  The number
// of pieces of a head is a power of two; the row of the j-th head is
// j / (2 kv_heads), by a multiplication that is exact for j < 2^20.)
template <int F>
struct Piece {
  static constexpr int E = F == FMT_F32 ? 4 : 8;           // elements of 16 bytes of activations
  int row, side, h, d;
  __device__ __forceinline__ Piece(const KvArgs &c, const KvIo &io, uint32_t i) {
    const uint32_t j = i >> io.piece_shift;
    row = (int)__umulhi(j, io.per_row);
    const int in = (int)j - row * 2 * c.kv_heads;
    side = in >= c.kv_heads;
    h = side ? in - c.kv_heads : in;
    d = (int)(i & ((1u << io.piece_shift) - 1u)) * E;
  }
};

constexpr int kBatch = 4;      // pieces of a thread in flight

template <int F, int R>
__global__ __launch_bounds__(256) void kv_write_kernel(KvArgs c, KvIo io) {
  __shared__ uint32_t place[R];
  const int row0 = io.first + blockIdx.x * R, rows = min(R, c.rows - row0);
  const int pieces = (rows * 2 * c.kv_heads) << io.piece_shift;
  // Four loads without a condition (past the end the last piece again), into vectors:
  // as structs behind a `break` the bf16 and fp32 ones went through LDS one by one
  // (8900 tokens 24.5 and 41.0 us).
  i32x4 u[kBatch];
  auto load = [&](int i0) MOE_INLINE {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const Piece<F> p(c, io, min(i0 + 256 * b + (int)threadIdx.x, pieces - 1));
      const long long at = (long long)(row0 + p.row) * (p.side ? io.v_row : io.k_row) +
                           p.h * (p.side ? io.v_head : io.k_head) + p.d;
      u[b] = *(const i32x4 *)((const uint8_t *)(p.side ? io.v : io.k) + at * (16 / Piece<F>::E));
    }
  };
  load(0);
  find_rows<R>(c, row0, place);
  __syncthreads();
  for (int i0 = 0; i0 < pieces; i0 += 256 * kBatch) {
    if (i0) load(i0);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + 256 * b + threadIdx.x;
      if (i >= pieces) continue;
      const Piece<F> p(c, io, i);
      const uint32_t at = place[p.row];
      if (at == kNoRow) continue;
      const long long dst = (long long)(at + ((uint32_t)p.h << c.page_shift)) * c.head_dim + p.d;
      uint8_t *pool = p.side ? c.v : c.k;
      if constexpr (F != FMT_MX8) {
        *(i32x4 *)(pool + dst * (16 / Piece<F>::E)) = u[b];
      } else {
        float v[8], am = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = __uint_as_float((uint32_t)u[b][j] << 16);
          v[2 * j + 1] = __uint_as_float((uint32_t)u[b][j] & 0xFFFF0000u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(v[j]));
        // four neighbouring lanes hold one block of 32 (a head's pieces are a
        // multiple of four, so a block's lanes agree on every condition above)
        am = fmaxf(am, __shfl_xor(am, 1, 64));
        am = fmaxf(am, __shfl_xor(am, 2, 64));
        const uint32_t sb = mx_scale_byte(am);
        const float inv = mx_inv_scale(sb);
        *(uint2 *)(pool + dst) =
            make_uint2(e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                       e4m3_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
        if ((threadIdx.x & 3) == 0) (p.side ? c.v_scale : c.k_scale)[dst >> 5] = (uint8_t)sb;
      }
    }
  }
}

template <int F, int R>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs c, KvIo io) {
  __shared__ uint32_t place[R];
  const int row0 = io.first + blockIdx.x * R, rows = min(R, c.rows - row0);
  const int pieces = (rows * 2 * c.kv_heads) << io.piece_shift;
  find_rows<R>(c, row0, place);
  __syncthreads();
  for (int i0 = 0; i0 < pieces; i0 += 256 * kBatch) {
    uint4 u[kBatch];
    uint32_t sb[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + 256 * b + threadIdx.x;
      u[b] = make_uint4(0, 0, 0, 0);
      sb[b] = 0;
      if (i >= pieces) break;
      const Piece<F> p(c, io, i);
      const uint32_t at = place[p.row];
      if (at == kNoRow) continue;
      const long long src = (long long)(at + ((uint32_t)p.h << c.page_shift)) * c.head_dim + p.d;
      const uint8_t *pool = p.side ? c.v : c.k;
      if constexpr (F == FMT_MX8) {
        const uint2 codes = *(const uint2 *)(pool + src);
        u[b].x = codes.x;
        u[b].y = codes.y;
        sb[b] = (p.side ? c.v_scale : c.k_scale)[src >> 5];
      } else {
        u[b] = *(const uint4 *)(pool + src * (16 / Piece<F>::E));
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + 256 * b + threadIdx.x;
      if (i >= pieces) break;
      const Piece<F> p(c, io, i);
      if constexpr (F == FMT_MX8) {
        const uint2 x = e4m3_to_bf16x4(u[b].x, sb[b]), y = e4m3_to_bf16x4(u[b].y, sb[b]);
        u[b] = make_uint4(x.x, x.y, y.x, y.y);
      }
      const long long out = ((long long)(row0 + p.row) * c.kv_heads + p.h) * c.head_dim + p.d;
      *(uint4 *)((uint8_t *)(p.side ? io.v : io.k) + out * (16 / Piece<F>::E)) = u[b];
    }
  }
}

namespace {
// Rows of a workgroup: 4 as long as all workgroups fit the chip at once (8 a
// CU), then 8: a second, nearly empty round of workgroups costs their whole
// latency again (8000 tokens of 8 heads of 128: 17 us with 4 rows, 12 with 8).
int rows_of_group(int rows) { return (rows + 3) / 4 <= 2048 ? 4 : 8; }

KvIo io_args(const KvArgs &c, void *k, void *v, long long k_row, long long k_head, long long v_row, long long v_head) {
  const int pieces = c.head_dim / (c.fmt == FMT_F32 ? 4 : 8);
  const uint64_t d = 2ull * c.kv_heads;
  return {k, v, k_row, k_head, v_row, v_head, __builtin_ctz(pieces), (uint32_t)(((1ull << 32) + d - 1) / d), 0};
}

// f(R, workgroups, io) for the rows of each launch.
template <typename Fn>
hipError_t each_launch(const KvArgs &c, KvIo io, Fn &&f) {
  constexpr int kRows = 1 << 25;
  static_assert(kRows / 4 <= max_groups(256), "rows of a launch");
  const int r = rows_of_group(c.rows);
  for (long long row0 = 0; row0 < c.rows; row0 += kRows) {
    io.first = (int)row0;
    const long long n = c.rows - row0 < kRows ? c.rows - row0 : kRows;
    f(r, (unsigned)((n + r - 1) / r), io);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <int F>
hipError_t write(const KvArgs &c, const KvIo &all, hipStream_t s) {
  return each_launch(c, all, [&](int r, unsigned grid, const KvIo &io) {
    if (r == 4) kv_write_kernel<F, 4><<<grid, 256, 0, s>>>(c, io);
    else kv_write_kernel<F, 8><<<grid, 256, 0, s>>>(c, io);
  });
}
template <int F>
hipError_t read(const KvArgs &c, const KvIo &all, hipStream_t s) {
  return each_launch(c, all, [&](int r, unsigned grid, const KvIo &io) {
    if (r == 4) kv_read_kernel<F, 4><<<grid, 256, 0, s>>>(c, io);
    else kv_read_kernel<F, 8><<<grid, 256, 0, s>>>(c, io);
  });
}
}  // namespace

hipError_t launch_kv_write(const KvArgs &c, const void *k, const void *v, long long k_row,
                           long long k_head, long long v_row, long long v_head, hipStream_t s) {
  if (c.rows <= 0) return hipSuccess;
  const KvIo io = io_args(c, const_cast<void *>(k), const_cast<void *>(v), k_row, k_head, v_row, v_head);
  return c.fmt == FMT_F32 ? write<FMT_F32>(c, io, s)
         : c.fmt == FMT_BF16 ? write<FMT_BF16>(c, io, s) : write<FMT_MX8>(c, io, s);
}

hipError_t launch_kv_read(const KvArgs &c, void *k, void *v, hipStream_t s) {
  if (c.rows <= 0) return hipSuccess;
  const KvIo io = io_args(c, k, v, 0, 0, 0, 0);
  return c.fmt == FMT_F32 ? read<FMT_F32>(c, io, s)
         : c.fmt == FMT_BF16 ? read<FMT_BF16>(c, io, s) : read<FMT_MX8>(c, io, s);
}

}  // namespace moe
