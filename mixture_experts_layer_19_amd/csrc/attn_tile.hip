// attn_tile.hip -- attention of chunks of new tokens over the paged cache.
//
// Bound by the matrix cores (bf16: 4 head_dim flops a row and key) and, next
// to them, by the LDS that feeds them and the exponentials.  A workgroup of
// four waves takes 128 QT query rows (tokens x heads of the group) and walks
// the keys in tiles of BK; a wave owns 32 QT rows.  S^T = K Q^T and
// O^T = V^T P^T on 32x32 matrix instructions: a lane holds scores of one query
// only, so the running maximum and sum are per lane (one exchange between the
// half waves), rescaling needs no other lane, and the weights are already the
// operand that the second product reads.
//
// K and V tiles come through registers (MX codes become bf16 there, exactly)
// into two LDS buffers: the loads of tile t + 1 run under the products of
// tile t, one barrier a tile.  Rows are XOR-swizzled in 16-byte chunks so that
// both reads, K's by rows and V's transposed, spread over the banks.
//
// The running maximum is a reference that moves only when a score passes it
// by 2^8: the weights stay below 2^8 of fp32 and the output is rescaled rarely.
//
// Few units: each is cut into `splits` runs of tiles, joined from the
// workspace in the order of their keys (attn_tile_join_kernel).
#include "attn_common.hpp"

namespace moe {

template <int F, int HD, int BK, int QT>
struct TileCfg {
  static constexpr int rows = 128 * QT;                    // query rows of a workgroup
  static constexpr int elem = F == FMT_F32 ? 4 : 2;        // in LDS
  static constexpr int row_bytes = HD * elem, chunks = row_bytes / 16;
  static constexpr int tile = BK * row_bytes;              // K or V
  static constexpr int lds = 4 * tile + 64;
  // staging of K or V, pieces of 16 bytes a thread: bf16 and fp32 by chunk, MX a run of
  // HD * BK / 256 codes of one key (under one scale)
  static constexpr int codes = HD * BK / 256;
  static constexpr int pieces = F == FMT_MX8 ? codes / 16 : tile / 16 / 256;
  static constexpr int QP = row_bytes / 32;                // 16-byte query pieces a lane
  static constexpr int KT = BK / 32, DT = HD / 32;
  // chunk c of key row r is stored at chunk c ^ swz(r)
  __device__ __forceinline__ static int swz(int r) {
    if constexpr (F == FMT_F32) return (r & 7) ^ (((r >> 2) & 1) << 3);
    else if constexpr (HD == 64) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    else return ((r & 3) << 2) | ((r >> 2) & 3);
  }
};

// Sequence and row tile of unit u, or s = -1 past the last unit.  The row
// tiles of a sequence come longest first.
template <int ROWS>
__device__ __forceinline__ void find_unit(const AttnArgs &a, int u, int &s, int &rt) {
  const int lane = threadIdx.x & 63;
  s = -1;
  rt = 0;
  for (int s0 = 0; s0 < a.c.seqs; s0 += 64) {
    int own = 0;
    if (s0 + lane < a.c.seqs)
      own = (int)(((long long)seq_geo(a.c, s0 + lane).n * a.group + ROWS - 1) / ROWS);
    int v = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int w = __shfl_up(v, d, 64);
      if (lane >= d) v += w;
    }
    const unsigned long long past = __ballot(v > u);
    if (past) {
      const int l = __ffsll((long long)past) - 1;
      s = s0 + l;
      rt = __shfl(v, l, 64) - 1 - u;               // descending
      return;
    }
    u -= __shfl(v, 63, 64);
  }
}

template <int F, int HD, int BK, int QT, int OCC>
__global__ __launch_bounds__(256, OCC) void attn_tile_kernel(AttnArgs a, int splits) {
  using C = TileCfg<F, HD, BK, QT>;
  constexpr int ROWS = C::rows, KT = C::KT, DT = C::DT, QP = C::QP, NP = C::pieces;
  extern __shared__ __align__(16) uint8_t lds[];           // K0 V0 K1 V1, flags
  int *flags = (int *)(lds + 4 * C::tile);                 // [stage][wave]
  const int tid = threadIdx.x, lane = tid & 63, q32 = lane & 31, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const KvArgs &c = a.c;

  const int h = blockIdx.x % c.kv_heads, split = blockIdx.x / c.kv_heads % splits;
  const int u = blockIdx.x / c.kv_heads / splits;
  int s, rt;
  find_unit<ROWS>(a, u, s, rt);
  s = __builtin_amdgcn_readfirstlane(s);
  if (s < 0) return clear_free_rows<F, HD>(a);
  const SeqGeo g = uniform(seq_geo(c, s));
  const int nrows = g.n * a.group, rt0 = __builtin_amdgcn_readfirstlane(rt) * ROWS;
  const int tok_a = rt0 / a.group, tok_b = (min(rt0 + ROWS, nrows) - 1) / a.group;
  const KeyRange<BK> range(g, tok_a, tok_b, a.window, a.sinks);
  const int per = (range.tiles + splits - 1) / splits;
  const int t0 = min(split * per, range.tiles), t1 = min(t0 + per, range.tiles);

  // queries: lane q32 holds row rt0 + 32 (QT wave + qt) + q32
  i32x4 q[QT][QP];
  int lo[QT], hi[QT];
  const int m0 = rt0 + 32 * QT * wave;
  static_for<QT>([&](auto qt) MOE_INLINE {
    const int m = m0 + 32 * qt + q32;
    const bool in = m < nrows;
    const int tok = in ? m / a.group : 0, hq = h * a.group + (in ? m % a.group : 0);
    const uint8_t *qp =
        (const uint8_t *)a.q + ((long long)(g.r0 + tok) * a.q_row + hq * a.q_head) * C::elem + 16 * hf;
#pragma unroll
    for (int p = 0; p < QP; ++p) q[qt][p] = in ? *(const i32x4 *)(qp + 32 * p) ^ (int)a.q_sign : i32x4{0, 0, 0, 0};
    const RowMask mask(g, tok, in, a.window, a.sinks);
    hi[qt] = mask.hi;
    lo[qt] = mask.lo;
  });
  // the wave's tokens; the keys that all, and that any, of its rows see
  const int wtok_a = m0 / a.group, wtok_b = (min(m0 + 32 * QT, nrows) - 1) / a.group;
  const bool has_rows = m0 < nrows;
  const int all_hi = min(g.pos0 + wtok_a + 1, g.len), any_hi = min(g.pos0 + wtok_b + 1, g.len);
  const int all_lo = a.window ? g.pos0 + wtok_b - a.window + 1 : 0;
  const int any_lo = a.window ? g.pos0 + wtok_a - a.window + 1 : 0;

  f32x16 o[QT][DT];
  float mx[QT], sum[QT];
#pragma unroll
  for (int qt = 0; qt < QT; ++qt) {
    mx[qt] = kNegBig;
    sum[qt] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[qt][d][i] = 0.0f;
  }

  // ---- staging
  const int32_t *pages = c.table + (long long)s * c.max_pages;
  // The table's entry for key `lane` of tile t, and the key's row in the pool.
  // As in the row kernel no load of the loop stands under a condition: past the
  // last tile, and for keys without a page, row 0 is read.
  auto page_of = [&](int t) MOE_INLINE {
    return pages[min((range.key(min(t, t1 - 1)) + (lane & (BK - 1))) >> c.page_shift, c.max_pages - 1)];
  };
  auto row_of = [&](int t, int page) MOE_INLINE {
    const int key = range.key(t) + (lane & (BK - 1));
    return t < t1 && key < g.len ? pool_row(c, page, h, key) : kNoRow;
  };
  // A tile's K or V on its way: K's is stored before V's is loaded, so that
  // both use the same registers.
  i32x4 st[NP];
  uint32_t st_scale = 0;
  // key of the tile that piece p of this thread belongs to
  auto piece_key = [&](int p) MOE_INLINE {
    if constexpr (F == FMT_MX8) return tid / (256 / BK);
    else return (p * 256 + tid) / C::chunks;
  };
  auto load_tile = [&](const uint8_t *pool, const uint8_t *scale, uint32_t row) MOE_INLINE {
    const uint32_t safe = row == kNoRow ? 0u : row;
    if constexpr (F == FMT_MX8) {
      const long long at = (long long)__shfl(safe, piece_key(0), 64) * HD + tid % (256 / BK) * C::codes;
#pragma unroll
      for (int p = 0; p < NP; ++p) st[p] = *(const i32x4 *)(pool + at + 16 * p);
      st_scale = scale[at >> 5];
    } else {
#pragma unroll
      for (int p = 0; p < NP; ++p)
        st[p] = *(const i32x4 *)(pool + (long long)__shfl(safe, piece_key(p), 64) * C::row_bytes +
                                 (p * 256 + tid) % C::chunks * 16);
    }
  };
  // (`finite`: zeros in place of what is not)
  auto put = [&](uint8_t *tile, auto finite) MOE_INLINE {
    auto chunk = [&](int key, int ch, uint4 w) MOE_INLINE {
      if constexpr (finite)
        w = make_uint4(word_finite<F>(w.x), word_finite<F>(w.y), word_finite<F>(w.z), word_finite<F>(w.w));
      *(uint4 *)(tile + key * C::row_bytes + ((ch ^ C::swz(key)) << 4)) = w;
    };
    if constexpr (F == FMT_MX8) {
      const int key = piece_key(0), part = tid % (256 / BK);
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint2 w0 = e4m3_to_bf16x4(st[p][2 * x], st_scale), w1 = e4m3_to_bf16x4(st[p][2 * x + 1], st_scale);
          chunk(key, part * (C::codes / 8) + 2 * p + x, make_uint4(w0.x, w0.y, w1.x, w1.y));
        }
    } else {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int id = p * 256 + tid;
        chunk(id / C::chunks, id % C::chunks, __builtin_bit_cast(uint4, st[p]));
      }
    }
  };
  // Tiles in which some of the workgroup's rows see a key that others do not.
  auto partial = [&](int t) MOE_INLINE {
    const int k0 = range.key(t);
    return tok_b > tok_a && (k0 + BK > g.pos0 + tok_a + 1 || (a.window && k0 <= g.pos0 + tok_b - a.window));
  };
  auto store_k = [&](int stage) MOE_INLINE { put(lds + 2 * stage * C::tile, std::false_type{}); };
  auto store_v = [&](int t, int stage, unsigned long long in) MOE_INLINE {
    if (in != ~0ull) {                                     // V of keys that do not exist: zeros
#pragma unroll
      for (int p = 0; p < NP; ++p)
        if (!((in >> piece_key(p)) & 1)) {
          st[p] = i32x4{0, 0, 0, 0};
          st_scale = 0;
        }
    }
    uint8_t *v = lds + (2 * stage + 1) * C::tile;
    if (partial(t)) {
      put(v, std::true_type{});
      bool bad = F == FMT_MX8 && st_scale >= kScaleOverflow;
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) bad = bad || word_not_finite<F>((uint32_t)st[p][i]);
      const unsigned long long any = __ballot(bad);
      if (lane == 0) flags[4 * stage + wave] = any != 0;
    } else {
      put(v, std::false_type{});
    }
  };

  // ---- products
  // K: lane q32 reads key row q32 of a 32-key tile, chunk 2 p + hf
  const uint32_t k_addr = q32 * C::row_bytes + ((hf ^ C::swz(q32)) << 4);
  // V: where this lane's first read lies; the swizzle makes the others' XORs of
  // it (added to a tile's offset, whose low bits are zero)
  const uint32_t v_addr =
      F == FMT_F32 ? 4 * hf * C::row_bytes + (((q32 >> 2) ^ C::swz(4 * hf)) << 4) + 4 * (q32 & 3)
                   : (4 * hf + ((lane & 15) >> 2)) * C::row_bytes + 8 * (lane & 1) +
                         (((2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ C::swz(4 * hf + ((lane & 15) >> 2))) << 4);
  auto scores = [&](int stage, f32x16 (&sc)[KT][QT]) MOE_INLINE {
    uint32_t addr = k_addr + 2 * stage * C::tile;
    asm volatile("" : "+v"(addr));                       // its XORs are cheaper than registers for them
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int qt = 0; qt < QT; ++qt)
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[kt][qt][i] = 0.0f;
    static_for<QP>([&](auto p) MOE_INLINE {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const i32x4 k = *(const i32x4 *)(lds + (addr ^ (32 * p)) + 32 * kt * C::row_bytes);
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
          if constexpr (F == FMT_F32) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sc[kt][qt] = __builtin_amdgcn_mfma_f32_32x32x2f32(__int_as_float(k[e]), __int_as_float(q[qt][p][e]),
                                                                sc[kt][qt], 0, 0, 0);
          } else {
            sc[kt][qt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8, k), __builtin_bit_cast(bf16x8, q[qt][p]), sc[kt][qt], 0, 0, 0);
          }
        }
      }
    });
    // K's reads run two pieces ahead of the products
    constexpr int PER = KT * QT * (F == FMT_F32 ? 4 : 1);
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * KT, 0);
    static_for<QP - 2>([&](auto) MOE_INLINE {
      __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, KT, 0);
    });
    __builtin_amdgcn_sched_group_barrier(0x008, 2 * PER, 0);
  };
  // O^T += V^T P^T for the 32 columns dt and the 32 keys kt.  The weights of
  // element i are those of key 8 (i / 4) + 4 hf + i % 4.
  auto add_pv = [&](uint32_t addr, int kt, int dt, const f32x16 (&p)[QT], const i32x4 (&pw)[QT][2]) MOE_INLINE {
    if constexpr (F == FMT_F32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = *(const float *)(lds + (addr ^ (16 * (i % 4)) ^ (128 * dt)) +
                                         (32 * kt + 8 * (i / 4) + i % 4) * C::row_bytes);
#pragma unroll
        for (int qt = 0; qt < QT; ++qt)
          o[qt][dt] = __builtin_amdgcn_mfma_f32_32x32x2f32(v, p[qt][i], o[qt][dt], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        s16x4 v[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          // a group of 16 lanes reads 4 keys x 16 columns, transposed
          using lds_s16x4 = __attribute__((address_space(3))) s16x4;
          v[b] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4 *)(lds + (addr ^ (64 * dt) ^ (32 * b)) + (32 * kt + 16 * st + 8 * b) * C::row_bytes));
        }
        const auto vv = __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int qt = 0; qt < QT; ++qt)
          o[qt][dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vv),
                                                             __builtin_bit_cast(bf16x8, pw[qt][st]), o[qt][dt], 0, 0, 0);
      }
    }
  };

  auto add_not_finite = [&](int k0) MOE_INLINE {
    int d0 = 4 * hf;
    asm volatile("" : "+v"(d0));                   // its addresses stay out of the loop's registers
    for (int key = k0; key < k0 + BK && key < g.len; ++key) {
      const uint32_t r = pool_row(c, pages[key >> c.page_shift], h, key);
      if (r == kNoRow) continue;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const f32x4 v = not_finite4<F, HD>(c, r, 32 * d + 8 * b + d0);
#pragma unroll
          for (int qt = 0; qt < QT; ++qt)
            if (key < hi[qt] && (key >= lo[qt] || key < a.sinks))
#pragma unroll
              for (int i = 0; i < 4; ++i) o[qt][d][4 * b + i] += v[i];
        }
    }
  };

  if (t0 < t1) {
    uint32_t row = row_of(t0, page_of(t0));
    unsigned long long there = __ballot(row != kNoRow);
    load_tile(c.k, c.k_scale, row);
    store_k(0);
    load_tile(c.v, c.v_scale, row);
    int page = page_of(t0 + 1);
    store_v(t0, 0, there);
    __syncthreads();
    for (int t = t0; t < t1; ++t) {
      const int stage = (t - t0) & 1, k0 = range.key(t);
      const unsigned long long there_now = there;
      row = row_of(t + 1, page);
      there = __ballot(row != kNoRow);
      load_tile(c.k, c.k_scale, row);
      __builtin_amdgcn_sched_barrier(0);
      const bool seen = has_rows && k0 < any_hi && (k0 + BK > any_lo || k0 < a.sinks);
      const bool inner = k0 + BK <= all_hi && (k0 >= all_lo || k0 + BK <= a.sinks) && there_now == ~0ull;
      f32x16 sc[KT][QT];
      if (seen) scores(stage, sc);
      __builtin_amdgcn_sched_barrier(0);
      store_k(stage ^ 1);
      load_tile(c.v, c.v_scale, row);
      page = page_of(t + 2);
      __builtin_amdgcn_sched_barrier(0);
      if (seen) {
        if (!inner) {
          static_for<KT>([&](auto kt) MOE_INLINE {
            uint32_t bits = (uint32_t)(there_now >> (32 * kt)) >> (4 * hf);
            asm volatile("" : "+v"(bits));                 // keeps the masks out of inner tiles
            const int base = k0 + 32 * kt + 4 * hf;
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
              const int below = hi[qt] - base, from = lo[qt] - base, sink = a.sinks - base;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int j = 8 * (i / 4) + i % 4;
                const bool see = ((bits >> j) & 1) && j < below && (j >= from || j < sink);
                sc[kt][qt][i] = see ? sc[kt][qt][i] : -INFINITY;
              }
            }
          });
        }
        i32x4 pw[KT][QT][2];
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
          float top = -INFINITY;
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[kt][qt][i]);
          top = max_half(top) * a.scale;                   // the scale is positive
          if (__ballot(top > mx[qt] + 8.0f)) {
            const float now = top > mx[qt] + 8.0f ? top : mx[qt];
            const float alpha = __builtin_amdgcn_exp2f(mx[qt] - now);
            mx[qt] = now;
            sum[qt] *= alpha;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int i = 0; i < 16; ++i) o[qt][d][i] *= alpha;
          }
          float part = 0.0f;
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float p = __builtin_amdgcn_exp2f(fmaf(sc[kt][qt][i], a.scale, -mx[qt]));
              sc[kt][qt][i] = p;
              part += p;
            }
            if constexpr (F != FMT_F32)
#pragma unroll
              for (int st = 0; st < 2; ++st)
                pw[kt][qt][st] = i32x4{(int)bf16_pack2(sc[kt][qt][8 * st], sc[kt][qt][8 * st + 1]),
                                       (int)bf16_pack2(sc[kt][qt][8 * st + 2], sc[kt][qt][8 * st + 3]),
                                       (int)bf16_pack2(sc[kt][qt][8 * st + 4], sc[kt][qt][8 * st + 5]),
                                       (int)bf16_pack2(sc[kt][qt][8 * st + 6], sc[kt][qt][8 * st + 7])};
          }
          sum[qt] += part;
        }
        uint32_t addr = v_addr + (2 * stage + 1) * C::tile;
        asm volatile("" : "+v"(addr));
        static_for<KT>([&](auto kt) MOE_INLINE {
          static_for<DT>([&](auto dt) MOE_INLINE { add_pv(addr, kt, dt, sc[kt], pw[kt]); });
        });
        if (partial(t) && (flags[4 * stage] | flags[4 * stage + 1] | flags[4 * stage + 2] | flags[4 * stage + 3]))
          add_not_finite(k0);
      }
      if (t + 1 < t1) store_v(t + 1, stage ^ 1, there);
      __syncthreads();
    }
  }

  // ---- results
#pragma unroll
  for (int qt = 0; qt < QT; ++qt) {
    const int m = m0 + 32 * qt + q32;
    const float l = sum_half(sum[qt]);
    if (m >= nrows) continue;
    if (splits == 1) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int tok = m / a.group, hq = h * a.group + m % a.group;
      const long long at = ((long long)(g.r0 + tok) * a.heads + hq) * HD + 4 * hf;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float v0 = o[qt][d][4 * b] * inv, v1 = o[qt][d][4 * b + 1] * inv;
          const float v2 = o[qt][d][4 * b + 2] * inv, v3 = o[qt][d][4 * b + 3] * inv;
          if constexpr (F == FMT_F32)
            *(f32x4 *)((float *)a.out + at + 32 * d + 8 * b) = f32x4{v0, v1, v2, v3};
          else
            *(uint2 *)((uint16_t *)a.out + at + 32 * d + 8 * b) = make_uint2(bf16_pack2(v0, v1), bf16_pack2(v2, v3));
        }
    } else {
      float *part = a.part + ((long long)u * c.kv_heads + h) * splits * ROWS * (HD + 2) +
                    (long long)split * ROWS * (HD + 2);
      const int r = m - rt0;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *(f32x4 *)(part + r * HD + 32 * d + 8 * b + 4 * hf) =
              f32x4{o[qt][d][4 * b], o[qt][d][4 * b + 1], o[qt][d][4 * b + 2], o[qt][d][4 * b + 3]};
      if (hf == 0) {
        part[ROWS * HD + 2 * r] = mx[qt];
        part[ROWS * HD + 2 * r + 1] = l;
      }
    }
  }
  clear_free_rows<F, HD>(a);
}

// Join the splits of a unit: HD / 4 threads a row, 4 columns each.
template <int F, int HD, int BK, int QT>
__global__ __launch_bounds__(256) void attn_tile_join_kernel(AttnArgs a, int splits) {
  constexpr int ROWS = TileCfg<F, HD, BK, QT>::rows, COLS = HD / 4, PER = 256 / COLS;
  const KvArgs &c = a.c;
  const int groups = ROWS / PER;                    // workgroups a unit
  const int gr = blockIdx.x % groups, h = blockIdx.x / groups % c.kv_heads, u = blockIdx.x / groups / c.kv_heads;
  int s, rt;
  find_unit<ROWS>(a, u, s, rt);
  if (s < 0) return;
  const SeqGeo g = seq_geo(c, s);
  const int r = gr * PER + threadIdx.x / COLS, col = threadIdx.x % COLS, m = rt * ROWS + r;
  if (m >= g.n * a.group) return;
  const float *part = a.part + ((long long)u * c.kv_heads + h) * splits * ROWS * (HD + 2);
  float top = kNegBig, l = 0.0f;
  for (int i = 0; i < splits; ++i) top = fmaxf(top, part[(long long)i * ROWS * (HD + 2) + ROWS * HD + 2 * r]);
  f32x4 acc = {0, 0, 0, 0};
  for (int i = 0; i < splits; ++i) {
    const float *p = part + (long long)i * ROWS * (HD + 2);
    const float e = __builtin_amdgcn_exp2f(p[ROWS * HD + 2 * r] - top);
    l += e * p[ROWS * HD + 2 * r + 1];
    acc += e * *(const f32x4 *)(p + r * HD + 4 * col);
  }
  acc *= l == 0.0f ? 0.0f : 1.0f / l;
  const int tok = m / a.group, hq = h * a.group + m % a.group;
  const long long at = ((long long)(g.r0 + tok) * a.heads + hq) * HD + 4 * col;
  if constexpr (F == FMT_F32)
    *(f32x4 *)((float *)a.out + at) = acc;
  else
    *(uint2 *)((uint16_t *)a.out + at) = make_uint2(bf16_pack2(acc[0], acc[1]), bf16_pack2(acc[2], acc[3]));
}

namespace {
template <int F, int HD, int BK, int QT, int OCC>
struct TileLaunch {
  using C = TileCfg<F, HD, BK, QT>;
  // row tiles of all sequences, at most
  static long long units(const AttnArgs &a) {
    const long long each = ((long long)a.c.max_rows * a.group + C::rows - 1) / C::rows * a.c.seqs;
    const long long all = (long long)a.c.rows * a.group / C::rows + a.c.seqs;
    return each < all ? each : all;
  }
  // Enough workgroups for every CU (OCC each), but four key tiles at least in
  // a run where the longest possible row sees that many.
  static int splits(const AttnArgs &a) {
    const long long wgs = units(a) * a.c.kv_heads, want = 256 * OCC;
    long long keys = (long long)a.c.max_pages << a.c.page_shift;
    if (a.window) {
      const long long seen = (long long)a.window + a.sinks + C::rows / a.group + 1;
      keys = keys < seen ? keys : seen;
    }
    const long long most = keys / (4 * BK) < 1 ? 1 : keys / (4 * BK);
    const long long s = want / wgs;
    return (int)(s < 1 ? 1 : s < most ? s : most);
  }
  static bool fits(const AttnArgs &a) {
    const long long u = units(a) * a.c.kv_heads;
    return u * splits(a) <= INT32_MAX && u * (C::rows / (1024 / HD)) <= INT32_MAX;
  }
  static size_t ws(const AttnArgs &a) {
    const int s = splits(a);
    return s == 1 ? 0 : (size_t)units(a) * a.c.kv_heads * s * C::rows * (HD + 2) * sizeof(float);
  }
  static hipError_t run(const AttnArgs &a, hipStream_t st) {
    const int s = splits(a);
    const long long u = units(a) * a.c.kv_heads, grid = u * s;
    static const hipError_t once = hipFuncSetAttribute((const void *)attn_tile_kernel<F, HD, BK, QT, OCC>,
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, C::lds);
    if (once != hipSuccess) return once;
    attn_tile_kernel<F, HD, BK, QT, OCC><<<(unsigned)grid, 256, C::lds, st>>>(a, s);
    if (s > 1)
      attn_tile_join_kernel<F, HD, BK, QT><<<(unsigned)(u * (C::rows / (1024 / HD))), 256, 0, st>>>(a, s);
    return hipGetLastError();
  }
};

template <typename Fn>
auto pick_tile(const KvArgs &c, Fn &&f) {
  if (c.fmt == FMT_F32) {
    if (c.head_dim == 64) return f(TileLaunch<FMT_F32, 64, 64, 1, 2>{});
    if (c.head_dim == 128) return f(TileLaunch<FMT_F32, 128, 32, 1, 1>{});
    return f(TileLaunch<FMT_F32, 256, 32, 1, 1>{});
  }
  if (c.fmt == FMT_BF16) {
    if (c.head_dim == 64) return f(TileLaunch<FMT_BF16, 64, 64, 1, 2>{});
    if (c.head_dim == 128) return f(TileLaunch<FMT_BF16, 128, 64, 1, 2>{});
    return f(TileLaunch<FMT_BF16, 256, 32, 1, 1>{});
  }
  if (c.head_dim == 64) return f(TileLaunch<FMT_MX8, 64, 64, 1, 2>{});
  if (c.head_dim == 128) return f(TileLaunch<FMT_MX8, 128, 64, 1, 2>{});
  return f(TileLaunch<FMT_MX8, 256, 32, 1, 1>{});
}
}  // namespace

size_t attn_tile_ws_bytes(const AttnArgs &a) {
  return pick_tile(a.c, [&](auto l) { return l.ws(a); });
}
bool attn_tile_fits(const AttnArgs &a) {
  return pick_tile(a.c, [&](auto l) { return l.fits(a); });
}
hipError_t launch_attn_tile(const AttnArgs &a, hipStream_t s) {
  return pick_tile(a.c, [&](auto l) { return l.run(a, s); });
}

}  // namespace moe
