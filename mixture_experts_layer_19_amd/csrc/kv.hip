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
// 132 (MX) or 256 on the other.  A workgroup takes a few rows; the row's
// place is looked up while its data is already on the way.
#include "block_common.hpp"

namespace moe {

struct KvIo {
  void *k, *v;                 // rows outside the pool
  long long k_row, k_head, v_row, v_head;
};

constexpr int kKvRows = 4;     // rows of a workgroup

// Place of each of the workgroup's rows in the pool, head 0 (kNoRow: none).
__device__ __forceinline__ void find_rows(const KvArgs &c, int row0, uint32_t *place) {
  const int wave = threadIdx.x >> 6;
  const int r = row0 + wave;
  uint32_t p = kNoRow;
  if (r < c.rows) {
    const int s = seq_of_row(c, r);
    if (s >= 0) {
      const SeqGeo g = seq_geo(c, s);
      const int pos = g.pos0 + (r - g.r0);
      if (r - g.r0 < g.n && pos >= 0 && pos < g.len)
        p = pool_row(c, c.table[(long long)s * c.max_pages + (pos >> c.page_shift)], 0, pos);
    }
  }
  if ((threadIdx.x & 63) == 0) place[wave] = p;
}

template <int F>
__global__ __launch_bounds__(256) void kv_write_kernel(KvArgs c, KvIo io) {
  __shared__ uint32_t place[kKvRows];
  const int row0 = blockIdx.x * kKvRows;
  find_rows(c, row0, place);
  __syncthreads();
  constexpr int E = F == FMT_F32 ? 4 : 8;        // elements of a 16-byte source piece
  const int per_head = c.head_dim / E, per_side = c.kv_heads * per_head;
  for (int i = threadIdx.x; i < kKvRows * 2 * per_side; i += 256) {
    const int rr = i / (2 * per_side), in = i % (2 * per_side), side = in / per_side;
    const int h = in % per_side / per_head, d = in % per_head * E, r = row0 + rr;
    if (r >= c.rows) break;
    const uint32_t at = place[rr];
    if (at == kNoRow) continue;
    const long long src = side ? r * io.v_row + h * io.v_head + d : r * io.k_row + h * io.k_head + d;
    const long long dst = (long long)(at + ((uint32_t)h << c.page_shift)) * c.head_dim + d;
    uint8_t *pool = side ? c.v : c.k;
    const void *from = side ? io.v : io.k;
    if constexpr (F == FMT_F32) {
      *(uint4 *)(pool + 4 * dst) = *(const uint4 *)((const float *)from + src);
    } else {
      const uint4 u = *(const uint4 *)((const uint16_t *)from + src);
      if constexpr (F == FMT_BF16) {
        *(uint4 *)(pool + 2 * dst) = u;
      } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float v[8], am = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = __uint_as_float(w[j] << 16);
          v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(v[j]));
        // four neighbouring lanes hold one block of 32 (the pieces of a row are
        // a multiple of four, so a block's lanes agree on every condition above)
        am = fmaxf(am, __shfl_xor(am, 1, 64));
        am = fmaxf(am, __shfl_xor(am, 2, 64));
        const uint32_t sb = mx_scale_byte(am);
        const float inv = mx_inv_scale(sb);
        *(uint2 *)(pool + dst) =
            make_uint2(e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                       e4m3_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
        if ((threadIdx.x & 3) == 0) (side ? c.v_scale : c.k_scale)[dst >> 5] = (uint8_t)sb;
      }
    }
  }
}

template <int F>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs c, KvIo io) {
  __shared__ uint32_t place[kKvRows];
  const int row0 = blockIdx.x * kKvRows;
  find_rows(c, row0, place);
  __syncthreads();
  constexpr int E = F == FMT_F32 ? 4 : 8;        // elements of a 16-byte output piece
  const int per_head = c.head_dim / E, per_side = c.kv_heads * per_head;
  for (int i = threadIdx.x; i < kKvRows * 2 * per_side; i += 256) {
    const int rr = i / (2 * per_side), in = i % (2 * per_side), side = in / per_side;
    const int h = in % per_side / per_head, d = in % per_head * E, r = row0 + rr;
    if (r >= c.rows) break;
    const uint32_t at = place[rr];
    const long long src = (long long)(at + ((uint32_t)h << c.page_shift)) * c.head_dim + d;
    const uint8_t *pool = side ? c.v : c.k;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (at != kNoRow) {
      if constexpr (F == FMT_F32) {
        u = *(const uint4 *)(pool + 4 * src);
      } else if constexpr (F == FMT_BF16) {
        u = *(const uint4 *)(pool + 2 * src);
      } else {
        const uint2 codes = *(const uint2 *)(pool + src);
        const uint32_t sb = (side ? c.v_scale : c.k_scale)[src >> 5];
        const uint2 a = e4m3_to_bf16x4(codes.x, sb), b = e4m3_to_bf16x4(codes.y, sb);
        u = make_uint4(a.x, a.y, b.x, b.y);
      }
    }
    const long long out = ((long long)r * c.kv_heads + h) * c.head_dim + d;
    *(uint4 *)((uint8_t *)(side ? io.v : io.k) + out * (F == FMT_F32 ? 4 : 2)) = u;
  }
}

hipError_t launch_kv_write(const KvArgs &c, const void *k, const void *v, long long k_row,
                           long long k_head, long long v_row, long long v_head, hipStream_t s) {
  if (c.rows <= 0) return hipSuccess;
  const KvIo io = {const_cast<void *>(k), const_cast<void *>(v), k_row, k_head, v_row, v_head};
  const unsigned grid = (unsigned)((c.rows + kKvRows - 1) / kKvRows);
  if (c.fmt == FMT_F32) kv_write_kernel<FMT_F32><<<grid, 256, 0, s>>>(c, io);
  else if (c.fmt == FMT_BF16) kv_write_kernel<FMT_BF16><<<grid, 256, 0, s>>>(c, io);
  else kv_write_kernel<FMT_MX8><<<grid, 256, 0, s>>>(c, io);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvArgs &c, void *k, void *v, hipStream_t s) {
  if (c.rows <= 0) return hipSuccess;
  const KvIo io = {k, v, 0, 0, 0, 0};
  const unsigned grid = (unsigned)((c.rows + kKvRows - 1) / kKvRows);
  if (c.fmt == FMT_F32) kv_read_kernel<FMT_F32><<<grid, 256, 0, s>>>(c, io);
  else if (c.fmt == FMT_BF16) kv_read_kernel<FMT_BF16><<<grid, 256, 0, s>>>(c, io);
  else kv_read_kernel<FMT_MX8><<<grid, 256, 0, s>>>(c, io);
  return hipGetLastError();
}

}  // namespace moe
