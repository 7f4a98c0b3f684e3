// attn_rows.hip -- attention of few query rows a sequence (single tokens, the
// few tokens of a speculative step) over the paged cache.
//
// Bound by memory: every key is read for at most 16 RT query rows.  So the
// work is split evenly over the chip along the keys: the tiles of all
// (sequence, KV head) units, laid end to end, are cut into one run of equal
// length a workgroup.  A workgroup that holds a whole unit writes its result;
// the pieces of a cut unit go to the workspace with their maximum and sum,
// and attn_join_kernel adds them in the order of their keys (no atomics: the
// result does not depend on timing).  The cut follows from the lengths on the
// device, so nothing is planned on the host and a captured graph follows
// lengths that change.
//
// Inside a workgroup the four waves take different keys, 16 NKH each, and
// need no barrier until their results are merged.  S^T = K Q^T and
// O^T = V^T P^T on 16x16 matrix instructions: with keys as the rows of S^T a
// lane holds scores of one query only, and they are already the operand that
// the second product reads.  K goes from memory straight to the registers the
// instruction reads; V goes through the wave's own LDS, read transposed.
//
// Measured, 64 heads over 8 KV heads of 128: 64 sequences of up to 8100 MX-fp8
// keys 114 us (5.1 TB/s), bf16 204 (5.5), 8 of up to 131071 bf16 keys 412 us (5.9
// TB/s), one of 937 bf16 keys 12 us, of which the join 4; fp32, up to 4000 keys,
// 209 us (5.4 TB/s); 32 sequences of 4 tokens over MX-fp8 74 us (4.0).
#include "attn_common.hpp"

namespace moe {

// Bytes of a pool row, and of the pieces of 16 that one lane of a 16-row
// fragment loads of it.  bf16, fp32: piece p at byte 64 p + 16 (l / 16), the
// same for K, V and Q.  MX: lane group g takes the quarter g of the row, so
// that its elements lie under one scale (two for head_dim 256).
template <int F, int HD>
struct RowFmt {
  static constexpr int elem = F == FMT_F32 ? 4 : F == FMT_BF16 ? 2 : 1;
  static constexpr int bytes = HD * elem, pieces = bytes / 64;
  static constexpr int q_elem = F == FMT_F32 ? 4 : 2, q_pieces = HD * q_elem / 64;
  // V in LDS: bf16 (read transposed, rows 32 bytes apart modulo the banks) or fp32
  static constexpr int v_pitch = F == FMT_F32 ? HD * 4 + 16 : HD * 2 + 32;
  static constexpr int scales = HD > 128 ? HD / 128 : 1;   // scale bytes a lane (MX)
};

template <int F, int HD, int RT, int NKH>
struct RowsCfg {
  using R = RowFmt<F, HD>;
  static constexpr int keys = 16 * NKH, BK = 4 * keys;     // a wave's, a workgroup's tile
  static constexpr int rows = 16 * RT;
  static constexpr int v_bytes = keys * R::v_pitch;        // a wave's V
  static constexpr int o_pitch = HD * 4 + 16, o_bytes = rows * o_pitch;
  static constexpr int wave_bytes = v_bytes > o_bytes ? v_bytes : o_bytes;
  static constexpr int lds = 4 * wave_bytes + 4 * rows * 8;
  // Cost of a unit, in tiles (Cut).  MX-fp8, 64 sequences of up to 8100 keys: 0
  // 122, 1 114, 2 115, 4 117 us; at head_dim 64: 74, 65, 63, 65; 32 sequences of 4
  // tokens (RT = 2): 80, 78, 71, 72; bf16, 64 sequences: 207, 202, 204, 210.
  static constexpr int unit_cost = RT == 2 || BK * R::bytes <= 8192 ? 2 : 1;
  // two workgroups a CU where the registers suffice: the one's loads run under
  // the other's products
  static constexpr int occupancy = RT == 1 && HD <= 128 ? 2 : 1;
};

// The even cut of the tiles of all units.  Unit order: sequence, row tile,
// KV head.  Every row tile of a sequence counts the sequence's tiles and, ahead
// of them, COST positions for what a unit costs beside them (lookups, the merge
// of its waves): a run of many short units would end last otherwise.
template <int BK, int ROWS, int COST>
struct Cut {
  const AttnArgs &a;
  int sums0;                   // scan(0)
  __device__ __forceinline__ Cut(const AttnArgs &args) : a(args), sums0(sums(0)) {}
  __device__ __forceinline__ static int row_tiles(const AttnArgs &a, const SeqGeo &g) {
    return (int)(((long long)g.n * a.group + ROWS - 1) / ROWS);
  }
  __device__ __forceinline__ static int tiles(const AttnArgs &a, const SeqGeo &g) {
    return max(KeyRange<BK>(g, 0, g.n - 1, a.window, a.sinks).tiles, 1);
  }
  // tiles of sequence s for one KV head
  __device__ __forceinline__ int weight(int s) const {
    if (s >= a.c.seqs) return 0;
    const SeqGeo g = seq_geo(a.c, s);
    return g.n ? row_tiles(a, g) * (tiles(a, g) + COST) : 0;
  }
  // inclusive sums of 64 sequences' weights from s0 on, one a lane
  __device__ __forceinline__ int sums(int s0) const {
    return wave_scan(weight(s0 + (threadIdx.x & 63)));
  }
  __device__ __forceinline__ int scan(int s0) const { return s0 ? sums(s0) : sums0; }
  __device__ __forceinline__ int total() const {
    int t = 0;
    for (int s0 = 0; s0 < a.c.seqs; s0 += 64) t += __builtin_amdgcn_readlane(scan(s0), 63);
    return t * a.c.kv_heads;
  }
  // sequence that holds position x, and the position of its first tile
  __device__ __forceinline__ int find(int x, int &start) const {
    int t = 0;
    for (int s0 = 0; s0 < a.c.seqs; s0 += 64) {
      const int v = scan(s0);
      const unsigned long long past = __ballot((t + v) * a.c.kv_heads > x);
      if (past) {
        const int l = __ffsll((long long)past) - 1;
        start = (t + (l ? __builtin_amdgcn_readlane(v, l - 1) : 0)) * a.c.kv_heads;
        return s0 + l;
      }
      t += __builtin_amdgcn_readlane(v, 63);
    }
    return -1;
  }
  // first position of sequence s
  __device__ __forceinline__ int first(int s) const {
    int t = 0;
    for (int s0 = 0; s0 < a.c.seqs; s0 += 64) {
      const int v = scan(s0);
      if (s < s0 + 64) return (t + (s > s0 ? __builtin_amdgcn_readlane(v, s - s0 - 1) : 0)) * a.c.kv_heads;
      t += __builtin_amdgcn_readlane(v, 63);
    }
    return t * a.c.kv_heads;
  }
};
struct NoCut {
  __device__ __forceinline__ NoCut(const AttnArgs &) {}
};
// The runs: the first `more` of them hold one tile more than the others.
struct Runs {
  int n, len, more;
  __device__ __forceinline__ Runs(int total, int grid)
      : n(min(grid, total)), len(n ? total / n : 0), more(n ? total % n : 0) {}
  __device__ __forceinline__ int start(int w) const { return w * len + min(w, more); }
  __device__ __forceinline__ int of(int x) const {
    const int cut = more * (len + 1);
    return x < cut ? x / (len + 1) : more + (x - cut) / len;
  }
};

// WHOLE: a workgroup a unit, nothing is cut (`units` row tiles a sequence).
template <int F, int HD, int RT, int NKH, bool WHOLE>
__global__ __launch_bounds__(256, (RowsCfg<F, HD, RT, NKH>::occupancy)) void attn_rows_kernel(AttnArgs a, int units) {
  using C = RowsCfg<F, HD, RT, NKH>;
  using R = typename C::R;
  constexpr int BK = C::BK, ROWS = C::rows, COST = C::unit_cost, DT = HD / 16;
  extern __shared__ __align__(16) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint8_t *own = lds + wave * C::wave_bytes;              // V, then O, of this wave
  float *ml = (float *)(lds + 4 * C::wave_bytes);          // [wave][row] maximum, sum
  const KvArgs &c = a.c;

  int x_begin = 0, x_end = 1;                              // this workgroup's run of tiles
  int whole_s = 0, whole_unit = 0;
  [[maybe_unused]] const std::conditional_t<WHOLE, NoCut, Cut<BK, ROWS, COST>> cut(a);
  if constexpr (WHOLE) {
    whole_s = blockIdx.x / (c.kv_heads * units);
    whole_unit = blockIdx.x % (c.kv_heads * units);
  } else {
    const Runs runs(__builtin_amdgcn_readfirstlane(cut.total()), a.grid);
    const bool idle = (int)blockIdx.x >= runs.n;
    x_begin = idle ? 0 : runs.start(blockIdx.x);
    x_end = idle ? 0 : runs.start(blockIdx.x + 1);
  }

  for (int x = x_begin; x < x_end;) {
    int s = whole_s, seq_x = 0;
    if constexpr (!WHOLE) s = __builtin_amdgcn_readfirstlane(cut.find(x, seq_x));
    const SeqGeo g = uniform(seq_geo(c, s));
    const KeyRange<BK> range(g, 0, g.n - 1, a.window, a.sinks);
    const int T = max(range.tiles, 1);
    const int in_seq = WHOLE ? 0 : x - __builtin_amdgcn_readfirstlane(seq_x);
    const int unit = WHOLE ? whole_unit : in_seq / (T + COST), at = WHOLE ? COST : in_seq % (T + COST);
    const int x_next = WHOLE ? x_end : min(x_end, x + (T + COST - at));
    const int t0 = max(at - COST, 0), t1 = WHOLE ? T : at + (x_next - x) - COST;
    if (t1 <= t0) break;                           // the run ends before the unit's tiles
    const int h = unit % c.kv_heads, rt0 = unit / c.kv_heads * ROWS;   // first row of the tile
    const int nrows = g.n * a.group;
    if (WHOLE && rt0 >= nrows) break;

    i32x4 q[RT][R::q_pieces];
    int lo[RT], hi[RT];
    f32x4 o[RT][DT];
    float mx[RT], sum[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      mx[rt] = kNegBig;
      sum[rt] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[rt][d] = f32x4{0, 0, 0, 0};
    }

    // The wave's tile t: its keys' entries of the table, their rows in the pool.
    // No load of the loop stands under a condition (past the last tile row 0 of
    // the pool is read again): with a load that may or may not have been issued,
    // waiting for an older one would be waiting for all.
    const int32_t *pages = c.table + (long long)s * c.max_pages;
    int page[NKH];
    auto load_pages = [&](int t) MOE_INLINE {
      const int k0 = range.key(min(t, t1 - 1)) + wave * C::keys;
#pragma unroll
      for (int kh = 0; kh < NKH; ++kh)
        page[kh] = pages[min((k0 + 16 * kh + l16) >> c.page_shift, c.max_pages - 1)];
    };
    uint32_t row[NKH];
    auto rows_of = [&](int t) MOE_INLINE {
      const int k0 = range.key(t) + wave * C::keys;
#pragma unroll
      for (int kh = 0; kh < NKH; ++kh) {
        const int key = k0 + 16 * kh + l16;
        row[kh] = t < t1 && key < g.len ? pool_row(c, page[kh], h, key) : kNoRow;
      }
    };
    i32x4 kr[NKH][R::pieces], vr[NKH][R::pieces];
    uint32_t ks[NKH][R::scales], vs[NKH][R::scales];
    auto load_rows = [&](const uint8_t *pool, const uint8_t *scale, i32x4 (&d)[NKH][R::pieces],
                         uint32_t (&sc)[NKH][R::scales]) MOE_INLINE {
#pragma unroll
      for (int kh = 0; kh < NKH; ++kh) {
        const long long r = row[kh] == kNoRow ? 0 : row[kh];
        const uint8_t *p = pool + r * R::bytes + (F == FMT_MX8 ? HD / 4 * g4 : 16 * g4);
#pragma unroll
        for (int i = 0; i < R::pieces; ++i)
          d[kh][i] = *(const i32x4 *)(p + (F == FMT_MX8 ? 16 * i : 64 * i));
        if constexpr (F == FMT_MX8) {
          const uint8_t *sp = scale + r * (HD / 32) + HD / 4 * g4 / 32;
#pragma unroll
          for (int i = 0; i < R::scales; ++i) sc[kh][i] = sp[i];
        }
      }
    };

    // V into this wave's LDS: [key][head_dim], bf16 or fp32
    // (`finite`: zeros in place of what is not)
    auto store_v = [&](auto finite) MOE_INLINE {
      auto put = [&](uint8_t *to, uint4 w) MOE_INLINE {
        if constexpr (finite)
          w = make_uint4(word_finite<F>(w.x), word_finite<F>(w.y), word_finite<F>(w.z), word_finite<F>(w.w));
        *(uint4 *)to = w;
      };
      static_for<NKH>([&](auto kh) MOE_INLINE {
        uint8_t *dst = own + (16 * kh + l16) * R::v_pitch;
        static_for<R::pieces>([&](auto p) MOE_INLINE {
          if constexpr (F == FMT_MX8) {
            constexpr int si = R::scales == 1 ? 0 : p / 2;
            uint8_t *to = dst + HD / 2 * g4 + 32 * p;
            const uint2 w0 = e4m3_to_bf16x4(vr[kh][p][0], vs[kh][si]);
            const uint2 w1 = e4m3_to_bf16x4(vr[kh][p][1], vs[kh][si]);
            const uint2 w2 = e4m3_to_bf16x4(vr[kh][p][2], vs[kh][si]);
            const uint2 w3 = e4m3_to_bf16x4(vr[kh][p][3], vs[kh][si]);
            put(to, make_uint4(w0.x, w0.y, w1.x, w1.y));
            put(to + 16, make_uint4(w2.x, w2.y, w3.x, w3.y));
          } else {
            put(dst + 64 * p + 16 * g4, __builtin_bit_cast(uint4, vr[kh][p]));
          }
        });
        if constexpr (F == FMT_MX8 && kh % 2 == 1) __builtin_amdgcn_sched_barrier(0);
      });
    };
    // The wave's LDS accesses before this point come before those after it.
    auto wave_sync = [&]() MOE_INLINE {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };
    f32x4 sc[RT][NKH];
    // O^T += V^T P^T, the weights in sc
    auto add_pv = [&]() MOE_INLINE {
      if constexpr (F == FMT_F32) {
        static_for<NKH>([&](auto kh) MOE_INLINE {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float *vp = (const float *)(own + (16 * kh + 4 * g4 + i) * R::v_pitch) + l16;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              const float v = vp[16 * d];
#pragma unroll
              for (int rt = 0; rt < RT; ++rt)
                o[rt][d] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, sc[rt][kh][i], o[rt][d], 0, 0, 0);
            }
          }
        });
      } else {
        static_for<NKH / 2>([&](auto kp) MOE_INLINE {
          i32x4 pw[RT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const f32x4 a0 = sc[rt][2 * kp], a1 = sc[rt][2 * kp + 1];
            pw[rt] = i32x4{(int)bf16_pack2(a0[0], a0[1]), (int)bf16_pack2(a0[2], a0[3]),
                           (int)bf16_pack2(a1[0], a1[1]), (int)bf16_pack2(a1[2], a1[3])};
          }
          // a group of 16 lanes reads 4 keys x 16 columns and gets, transposed, one
          // column of 4 keys a lane: keys 4 g4 .. of each half
          uint8_t *vp = own + (32 * kp + 4 * g4 + (l16 >> 2)) * R::v_pitch + 8 * (l16 & 3);
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            using lds_s16x4 = __attribute__((address_space(3))) s16x4;
            const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vp + 32 * d));
            const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vp + 32 * d + 16 * R::v_pitch));
            const auto v = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              o[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, pw[rt]), o[rt][d], 0, 0, 0);
          }
        });
      }
    };
    auto add_not_finite = [&](int k0) MOE_INLINE {
      int d0 = 4 * g4;
      asm volatile("" : "+v"(d0));                 // its addresses stay out of the loop's registers
      for (int key = k0; key < k0 + C::keys && key < g.len; ++key) {
        const uint32_t r = pool_row(c, pages[key >> c.page_shift], h, key);
        if (r == kNoRow) continue;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const f32x4 v = not_finite4<F, HD>(c, r, 16 * d + d0);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            if (key < hi[rt] && (key >= lo[rt] || key < a.sinks)) o[rt][d] += v;
        }
      }
    };
    auto clear_v = [&](i32x4 (&d)[R::pieces], uint32_t (&sb)[R::scales]) MOE_INLINE {
#pragma unroll
      for (int p = 0; p < R::pieces; ++p) d[p] = i32x4{0, 0, 0, 0};
      if constexpr (F == FMT_MX8)
#pragma unroll
        for (int i = 0; i < R::scales; ++i) sb[i] = 0;
    };
    // Whether any element is infinite or NaN, or (MX) may be so in bf16.
    auto not_finite = [&](const i32x4 (&d)[R::pieces], const uint32_t (&sb)[R::scales]) MOE_INLINE {
      bool bad = false;
#pragma unroll
      for (int p = 0; p < R::pieces; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          bad = bad || word_not_finite<F>((uint32_t)d[p][i]);
      if constexpr (F == FMT_MX8)
#pragma unroll
        for (int i = 0; i < R::scales; ++i) bad = bad || sb[i] >= kScaleOverflow;
      return bad;
    };
    // tokens of the row tile, and the keys that all of them see
    const int tok_a = rt0 / a.group, tok_b = (min(rt0 + ROWS, nrows) - 1) / a.group;
    const int all_hi = min(g.pos0 + tok_a + 1, g.len), all_lo = a.window ? g.pos0 + tok_b - a.window + 1 : 0;

    load_pages(t0);
    __builtin_amdgcn_sched_barrier(0);
    // queries: lane l16 holds row rt0 + 16 rt + l16
    static_for<RT>([&](auto rt) MOE_INLINE {
      const int m = rt0 + 16 * rt + l16;
      const bool in = m < nrows;
      const int tok = in ? m / a.group : 0, hq = h * a.group + (in ? m % a.group : 0);
      const uint8_t *qp = (const uint8_t *)a.q +
                          ((long long)(g.r0 + tok) * a.q_row + hq * a.q_head) * R::q_elem;
#pragma unroll
      for (int p = 0; p < R::q_pieces; ++p) {
        const int off = F == FMT_MX8 ? HD / 2 * g4 + 16 * p : 64 * p + 16 * g4;
        q[rt][p] = in ? *(const i32x4 *)(qp + off) ^ (int)a.q_sign : i32x4{0, 0, 0, 0};
      }
      const RowMask mask(g, tok, in, a.window, a.sinks);
      hi[rt] = mask.hi;
      lo[rt] = mask.lo;
    });

    // in the loop's order: its waits count the loads issued since
    rows_of(t0);
    load_rows(c.k, c.k_scale, kr, ks);
    __builtin_amdgcn_sched_barrier(0);
    load_pages(t0 + 1);
    __builtin_amdgcn_sched_barrier(0);
    load_rows(c.v, c.v_scale, vr, vs);
    __builtin_amdgcn_sched_barrier(0);

    for (int t = t0; t < t1; ++t) {
      const int k0 = range.key(t) + wave * C::keys;
      // keys that exist: bit l of half kh is key k0 + 16 kh + l
      uint32_t there[NKH];
      bool all = true;
#pragma unroll
      for (int kh = 0; kh < NKH; ++kh) {
        const unsigned long long m = __ballot(row[kh] != kNoRow);
        there[kh] = (uint32_t)m & 0xFFFFu;
        all = all && there[kh] == 0xFFFFu;
      }
      // S^T = K Q^T: lane l16 holds row l16 of the queries, keys 16 kh + 4 g4 + i
      static_for<NKH>([&](auto kh) MOE_INLINE {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sc[rt][kh] = f32x4{0, 0, 0, 0};
        static_for<R::pieces>([&](auto p) MOE_INLINE {
          if constexpr (F == FMT_MX8) {
            constexpr int si = R::scales == 1 ? 0 : p / 2;
            const uint2 w0 = e4m3_to_bf16x4(kr[kh][p][0], ks[kh][si]);
            const uint2 w1 = e4m3_to_bf16x4(kr[kh][p][1], ks[kh][si]);
            const uint2 w2 = e4m3_to_bf16x4(kr[kh][p][2], ks[kh][si]);
            const uint2 w3 = e4m3_to_bf16x4(kr[kh][p][3], ks[kh][si]);
            const uint4 lo8 = make_uint4(w0.x, w0.y, w1.x, w1.y), hi8 = make_uint4(w2.x, w2.y, w3.x, w3.y);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              sc[rt][kh] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, lo8), __builtin_bit_cast(bf16x8, q[rt][2 * p]), sc[rt][kh], 0, 0, 0);
              sc[rt][kh] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, hi8), __builtin_bit_cast(bf16x8, q[rt][2 * p + 1]), sc[rt][kh], 0, 0, 0);
            }
          } else if constexpr (F == FMT_BF16) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              sc[rt][kh] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, kr[kh][p]), __builtin_bit_cast(bf16x8, q[rt][p]), sc[rt][kh], 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int rt = 0; rt < RT; ++rt)
                sc[rt][kh] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                    __int_as_float(kr[kh][p][e]), __int_as_float(q[rt][p][e]), sc[rt][kh], 0, 0, 0);
          }
        });
        // codes of two halves at a time become bf16: more would not fit the registers
        if constexpr (F == FMT_MX8 && kh % 2 == 1) __builtin_amdgcn_sched_barrier(0);
      });
      __builtin_amdgcn_sched_barrier(0);
      rows_of(t + 1);
      load_rows(c.k, c.k_scale, kr, ks);
      __builtin_amdgcn_sched_barrier(0);
      // before V's loads: waiting for the pages, which the next K needs, is then
      // not waiting for V
      load_pages(t + 2);
      __builtin_amdgcn_sched_barrier(0);

      // softmax over the tile; sc becomes the weights
      const bool inner = all && k0 + C::keys <= all_hi && (k0 >= all_lo || k0 + C::keys <= a.sinks);
      if (!inner) {
#pragma unroll
        for (int kh = 0; kh < NKH; ++kh) {
          uint32_t bits = there[kh];
          asm volatile("" : "+v"(bits));           // keeps the masks out of inner tiles
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 4 * g4 + i, key = k0 + 16 * kh + j;
              const bool see = ((bits >> j) & 1) && key < hi[rt] && (key >= lo[rt] || key < a.sinks);
              sc[rt][kh][i] = see ? sc[rt][kh][i] : -INFINITY;
            }
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float top = -INFINITY;
#pragma unroll
        for (int kh = 0; kh < NKH; ++kh)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[rt][kh][i]);
        top = max_rows16(top) * a.scale;           // the scale is positive
        // the reference moves only when a score passes it by 2^8
        if (__ballot(top > mx[rt] + 8.0f)) {
          const float now = top > mx[rt] + 8.0f ? top : mx[rt];
          const float alpha = __builtin_amdgcn_exp2f(mx[rt] - now);
          mx[rt] = now;
          sum[rt] *= alpha;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[rt][d] *= alpha;
        }
        float part = 0.0f;
#pragma unroll
        for (int kh = 0; kh < NKH; ++kh)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = __builtin_amdgcn_exp2f(mul_sub(sc[rt][kh][i], a.scale, mx[rt]));
            sc[rt][kh][i] = p;
            part += p;
          }
        sum[rt] += part;
      }

      // V of keys that do not exist: zeros (their weight is zero, but zero times
      // what a free page holds need not be)
      if (!all)
        static_for<NKH>([&](auto kh) MOE_INLINE {
          if (!((there[kh] >> l16) & 1)) clear_v(vr[kh], vs[kh]);
        });
      // keys that exist and that not all rows see (of a single token too: behind its
      // window, past its sinks)
      bool unsafe = false;
      if (min(k0 + C::keys, g.len) > all_hi || (k0 < all_lo && k0 + C::keys > a.sinks))
        static_for<NKH>([&](auto kh) MOE_INLINE { unsafe = unsafe || not_finite(vr[kh], vs[kh]); });
      const bool fix = __ballot(unsafe) != 0;
      if (fix) store_v(std::true_type{});
      else store_v(std::false_type{});
      __builtin_amdgcn_sched_barrier(0);
      load_rows(c.v, c.v_scale, vr, vs);
      wave_sync();
      add_pv();
      if (fix) add_not_finite(k0);
      wave_sync();
    }

    // merge the four waves: O [row][head_dim], maximum and sum of each row
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float l = sum_rows16(sum[rt]);
#pragma unroll
      for (int d = 0; d < DT; ++d)
        *(f32x4 *)(own + (16 * rt + l16) * C::o_pitch + (16 * d + 4 * g4) * 4) = o[rt][d];
      if (g4 == 0) {
        ml[(wave * ROWS + 16 * rt + l16) * 2] = mx[rt];
        ml[(wave * ROWS + 16 * rt + l16) * 2 + 1] = l;
      }
    }
    __syncthreads();
    const bool whole = WHOLE || (t0 == 0 && t1 == T);
    // a run holds at most two cut units: one it starts inside of, one it ends inside of
    const long long slot = 2ll * blockIdx.x + (x == x_begin ? 0 : 1);
    float *part = a.part + slot * ROWS * (HD + 2);
    for (int i = tid; i < ROWS * HD / 4; i += 256) {
      const int m = i / (HD / 4), d = i % (HD / 4) * 4;
      if (rt0 + m >= nrows) break;
      float top = kNegBig, l = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[(w * ROWS + m) * 2]);
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float e = __builtin_amdgcn_exp2f(ml[(w * ROWS + m) * 2] - top);
        l += e * ml[(w * ROWS + m) * 2 + 1];
        acc += e * *(const f32x4 *)(lds + w * C::wave_bytes + m * C::o_pitch + d * 4);
      }
      if (whole) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        acc *= inv;
        const int tok = (rt0 + m) / a.group, hq = h * a.group + (rt0 + m) % a.group;
        const long long at = ((long long)(g.r0 + tok) * a.heads + hq) * HD + d;
        if constexpr (F == FMT_F32)
          *(f32x4 *)((float *)a.out + at) = acc;
        else
          *(uint2 *)((uint16_t *)a.out + at) =
              make_uint2(bf16_pack2(acc[0], acc[1]), bf16_pack2(acc[2], acc[3]));
      } else {
        *(f32x4 *)(part + m * HD + d) = acc;
        if (d == 0) {
          part[ROWS * HD + 2 * m] = top;
          part[ROWS * HD + 2 * m + 1] = l;
        }
      }
    }
    __syncthreads();
    x = x_next;
  }
  clear_free_rows<F, HD>(a);
}

// Join the pieces of cut units, 4 columns a thread.  With few units a
// workgroup takes one row (`per` = 1), its 256 / COLS groups of threads every
// SL-th piece each; with many it takes SL rows (`per` = SL), one a group, since
// a unit then has few pieces.
template <int F, int HD, int RT, int NKH>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int unit_rows, int units, int per) {
  using C = RowsCfg<F, HD, RT, NKH>;
  constexpr int BK = C::BK, ROWS = C::rows, COST = C::unit_cost;
  constexpr int COLS = HD / 4, SL = 256 / COLS;
  __shared__ f32x4 red[256];
  __shared__ float redm[SL][2];
  const KvArgs &c = a.c;
  const int tid = threadIdx.x, col = tid % COLS, sl = tid / COLS;
  const int parts = (unit_rows + per - 1) / per;
  const int unit = blockIdx.x / parts, h = unit % c.kv_heads;
  const int s = unit / c.kv_heads / units, rt = unit / c.kv_heads % units;
  const int m = blockIdx.x % parts * per + (per == 1 ? 0 : sl);
  const Cut<BK, ROWS, COST> cut(a);
  const SeqGeo g = uniform(seq_geo(c, s));
  const int nrows = g.n * a.group - rt * ROWS;      // of this unit
  if (nrows <= 0) return;
  const Runs runs(__builtin_amdgcn_readfirstlane(cut.total()), a.grid);
  const int T = Cut<BK, ROWS, COST>::tiles(a, g);
  const int x0 = __builtin_amdgcn_readfirstlane(cut.first(s)) + (rt * c.kv_heads + h) * (T + COST);
  const int w0 = runs.of(x0 + COST), w1 = runs.of(x0 + COST + T - 1);
  if (w0 == w1) return;                            // never cut: its workgroup wrote it
  const int first_slot = 2 * w0 + (runs.start(w0) >= x0 ? 0 : 1);
  const bool in = m < min(nrows, ROWS) && m < unit_rows;
  const int mr = in ? m : 0;
  float top = kNegBig, l = 0.0f;
  f32x4 acc = {0, 0, 0, 0};
  constexpr int AHEAD = 4;                         // pieces in flight a thread
  const int step = per == 1 ? SL : 1;
  for (int w = w0 + (per == 1 ? sl : 0); w <= w1; w += AHEAD * step) {
    float pm[AHEAD], pl[AHEAD];
    f32x4 po[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int wi = min(w + i * step, w1);
      const float *p = a.part + (long long)(wi == w0 ? first_slot : 2 * wi) * ROWS * (HD + 2);
      pm[i] = p[ROWS * HD + 2 * mr];
      pl[i] = p[ROWS * HD + 2 * mr + 1];
      po[i] = *(const f32x4 *)(p + mr * HD + 4 * col);
    }
    float nt = top;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) nt = fmaxf(nt, w + i * step <= w1 ? pm[i] : kNegBig);
    const float e0 = __builtin_amdgcn_exp2f(top - nt);
    acc *= e0;
    l *= e0;
    top = nt;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (w + i * step <= w1) {
        const float e = __builtin_amdgcn_exp2f(pm[i] - nt);
        acc += po[i] * e;
        l += pl[i] * e;
      }
  }
  if (per == 1) {
    red[tid] = acc;
    if (col == 0) { redm[sl][0] = top; redm[sl][1] = l; }
    __syncthreads();
    if (sl) return;
    top = kNegBig;
    l = 0.0f;
    acc = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < SL; ++i) top = fmaxf(top, redm[i][0]);
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const float e = __builtin_amdgcn_exp2f(redm[i][0] - top);
      l += e * redm[i][1];
      acc += e * red[i * COLS + col];
    }
  }
  if (!in) return;
  acc *= l == 0.0f ? 0.0f : 1.0f / l;
  const int tok = (rt * ROWS + m) / a.group, hq = h * a.group + (rt * ROWS + m) % a.group;
  const long long at = ((long long)(g.r0 + tok) * a.heads + hq) * HD + 4 * col;
  if constexpr (F == FMT_F32)
    *(f32x4 *)((float *)a.out + at) = acc;
  else
    *(uint2 *)((uint16_t *)a.out + at) = make_uint2(bf16_pack2(acc[0], acc[1]), bf16_pack2(acc[2], acc[3]));
}

namespace {
// Two workgroups a CU.  More, where the registers hold them, cut more units: MX-fp8
// at head_dim 64, 64 sequences of up to 8100 keys, 60 us against 63 (three) and 64.
constexpr int kRowsGrid = 512;

template <int F, int HD, int RT, int NKH>
struct Launch {
  using C = RowsCfg<F, HD, RT, NKH>;
  static int units(const KvArgs &c, int group) {   // row tiles of the longest sequence
    return (int)(((long long)c.max_rows * group + C::rows - 1) / C::rows);
  }
  // tiles of all units, at most; -1 past 32 bits, which the kernels count in
  static long long most(const KvArgs &c, int group) {
    const long long tiles = (((long long)c.max_pages << c.page_shift) + C::BK - 1) / C::BK + 1 + C::unit_cost;
    const long long sums = tiles * units(c, group);
    if (sums > INT32_MAX) return -1;
    const long long seq = sums * c.kv_heads;
    return seq > INT32_MAX || seq * c.seqs > INT32_MAX ? -1 : seq * c.seqs;
  }
  static int grid(const KvArgs &c, int group) {
    const long long all = most(c, group);
    return (int)(all >= 0 && all < kRowsGrid ? all : kRowsGrid);
  }
  // Up to six tiles a unit (768 keys of bf16 and MX) are not cut: to walk them
  // costs less than the second launch that joins their pieces (one sequence of
  // 600 keys: 12.9 us against 14.5; 30 of up to 480: 10.1 against 19.3; one of
  // 937, eight tiles: 17.6 against 13.9).
  static bool whole(const AttnArgs &a) {
    long long tiles = (((long long)a.c.max_pages << a.c.page_shift) + C::BK - 1) / C::BK;
    if (a.window) {
      const long long seen = (a.window + (long long)a.c.max_rows - 2) / C::BK + 2 + (a.sinks + C::BK - 1) / C::BK;
      tiles = tiles < seen ? tiles : seen;
    }
    return tiles <= 6;
  }
  // Units, and what the join's launch holds of them: rows of a unit, at most, and
  // how many of them a workgroup takes.
  static long long all_units(const KvArgs &c, int group) { return (long long)c.seqs * c.kv_heads * units(c, group); }
  static int unit_rows(const AttnArgs &a) {
    const long long rows = (long long)a.c.max_rows * a.group;
    return (int)(rows < C::rows ? rows : C::rows);
  }
  static int per(const AttnArgs &a) { return all_units(a.c, a.group) < 256 ? 1 : 1024 / HD; }
  static long long join_groups(const AttnArgs &a) {
    return all_units(a.c, a.group) * ((unit_rows(a) + per(a) - 1) / per(a));
  }
  static bool fits(const AttnArgs &a) {
    return most(a.c, a.group) >= 0 && (whole(a) ? all_units(a.c, a.group) : join_groups(a)) <= max_groups(256);
  }
  static size_t ws(const AttnArgs &a) {
    return whole(a) ? 0 : (size_t)grid(a.c, a.group) * 2 * C::rows * (HD + 2) * sizeof(float);
  }
  template <bool WHOLE>
  static hipError_t rows(const AttnArgs &a, int u, hipStream_t s) {
    static OncePerDevice once;
    const hipError_t err = allow_lds(once, (const void *)attn_rows_kernel<F, HD, RT, NKH, WHOLE>, C::lds);
    if (err != hipSuccess) return err;
    attn_rows_kernel<F, HD, RT, NKH, WHOLE><<<a.grid, 256, C::lds, s>>>(a, u);
    return hipGetLastError();
  }
  static hipError_t run(const AttnArgs &args, hipStream_t s) {
    AttnArgs a = args;
    const int u = units(a.c, a.group);
    if (whole(a)) {
      a.grid = (int)all_units(a.c, a.group);
      return rows<true>(a, u, s);
    }
    a.grid = grid(a.c, a.group);
    const hipError_t err = rows<false>(a, u, s);
    if (err != hipSuccess) return err;
    attn_join_kernel<F, HD, RT, NKH><<<(unsigned)join_groups(a), 256, 0, s>>>(a, unit_rows(a), u, per(a));
    return hipGetLastError();
  }
};

// f(Launch<...>{}) of the variant for this cache and number of rows a sequence
template <typename Fn>
auto pick(const KvArgs &c, int group, Fn &&f) {
  const bool one = (long long)c.max_rows * group <= 16;   // else 32 rows a tile
#define MOE_PICK(F, HD, NKH) return one ? f(Launch<F, HD, 1, NKH>{}) : f(Launch<F, HD, 2, NKH>{})
  if (c.fmt == FMT_F32) {
    if (c.head_dim == 64) MOE_PICK(FMT_F32, 64, 2);
    if (c.head_dim == 128) MOE_PICK(FMT_F32, 128, 1);
    return f(Launch<FMT_F32, 256, 1, 1>{});        // 32 rows of fp32 at 256 do not fit the registers
  }
  if (c.fmt == FMT_BF16) {
    if (c.head_dim == 64) MOE_PICK(FMT_BF16, 64, 2);
    if (c.head_dim == 128) MOE_PICK(FMT_BF16, 128, 2);
    MOE_PICK(FMT_BF16, 256, 2);
  }
  if (c.head_dim == 64) MOE_PICK(FMT_MX8, 64, 2);
  if (c.head_dim == 128) MOE_PICK(FMT_MX8, 128, 2);
  MOE_PICK(FMT_MX8, 256, 2);
#undef MOE_PICK
}
}  // namespace

size_t attn_rows_ws_bytes(const AttnArgs &a) {
  return pick(a.c, a.group, [&](auto l) { return l.ws(a); });
}
bool attn_rows_fits(const AttnArgs &a) {
  return pick(a.c, a.group, [&](auto l) { return l.fits(a); });
}
hipError_t launch_attn_rows(const AttnArgs &a, hipStream_t s) {
  return pick(a.c, a.group, [&](auto l) { return l.run(a, s); });
}

}  // namespace moe
