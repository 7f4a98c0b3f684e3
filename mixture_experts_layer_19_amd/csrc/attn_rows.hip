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
};

// The even cut of the tiles of all units.  Unit order: sequence, row tile,
// KV head.  Every row tile of a sequence counts the sequence's tiles.
template <int BK, int ROWS>
struct Cut {
  const AttnArgs &a;
  __device__ __forceinline__ Cut(const AttnArgs &args) : a(args) {}
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
    return g.n ? row_tiles(a, g) * tiles(a, g) : 0;
  }
  // inclusive sums of 64 sequences' weights from s0 on, one a lane
  __device__ __forceinline__ int scan(int s0) const {
    const int lane = threadIdx.x & 63;
    int v = weight(s0 + lane);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(v, d, 64);
      if (lane >= d) v += u;
    }
    return v;
  }
  __device__ __forceinline__ long long total() const {
    long long t = 0;
    for (int s0 = 0; s0 < a.c.seqs; s0 += 64) t += __shfl(scan(s0), 63, 64);
    return t * a.c.kv_heads;
  }
  // sequence that holds position x, and the position of its first tile
  __device__ __forceinline__ int find(long long x, long long &start) const {
    long long t = 0;
    for (int s0 = 0; s0 < a.c.seqs; s0 += 64) {
      const int v = scan(s0);
      const int sum = __shfl(v, 63, 64);
      if ((t + sum) * a.c.kv_heads > x) {
        const unsigned long long past = __ballot((t + v) * a.c.kv_heads > x);
        const int l = __ffsll((long long)past) - 1;
        start = (t + (l ? __shfl(v, l - 1, 64) : 0)) * a.c.kv_heads;
        return s0 + l;
      }
      t += sum;
    }
    return -1;
  }
  // first position of sequence s
  __device__ __forceinline__ long long first(int s) const {
    long long t = 0;
    for (int s0 = 0; s0 < a.c.seqs; s0 += 64) {
      const int v = scan(s0);
      if (s < s0 + 64) return (t + (s > s0 ? __shfl(v, s - s0 - 1, 64) : 0)) * a.c.kv_heads;
      t += __shfl(v, 63, 64);
    }
    return t * a.c.kv_heads;
  }
};
// first position of workgroup w's run; the workgroup that holds position x
__device__ __forceinline__ long long run_start(long long total, int w, int runs) { return total * w / runs; }
__device__ __forceinline__ int run_of(long long total, long long x, int runs) {
  int w = (int)(x * runs / total);
  while (w + 1 < runs && run_start(total, w + 1, runs) <= x) ++w;
  while (w > 0 && run_start(total, w, runs) > x) --w;
  return w;
}

template <int F, int HD, int RT, int NKH>
__global__ __launch_bounds__(256) void attn_rows_kernel(AttnArgs a) {
  using C = RowsCfg<F, HD, RT, NKH>;
  using R = typename C::R;
  constexpr int BK = C::BK, ROWS = C::rows, DT = HD / 16;
  extern __shared__ __align__(16) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint8_t *own = lds + wave * C::wave_bytes;              // V, then O, of this wave
  float *ml = (float *)(lds + 4 * C::wave_bytes);          // [wave][row] maximum, sum
  const KvArgs &c = a.c;

  const Cut<BK, ROWS> cut(a);
  const long long total = cut.total();
  const int runs = (int)min((long long)a.grid, total);     // no run is empty
  if ((int)blockIdx.x >= runs) return;
  long long x = run_start(total, blockIdx.x, runs);
  const long long x_begin = x, x_end = run_start(total, blockIdx.x + 1, runs);

  while (x < x_end) {
    long long seq_x;
    const int s = __builtin_amdgcn_readfirstlane(cut.find(x, seq_x));
    const SeqGeo g = seq_geo(c, s);
    const KeyRange<BK> range(g, 0, g.n - 1, a.window, a.sinks);
    const int T = max(range.tiles, 1);
    const int unit = (int)((x - seq_x) / T), t0 = (int)((x - seq_x) % T);
    const int t1 = (int)min((long long)T, t0 + (x_end - x));
    const int h = unit % c.kv_heads, rt0 = unit / c.kv_heads * ROWS;   // first row of the tile
    const int nrows = g.n * a.group;

    // queries: lane l16 holds row rt0 + 16 rt + l16
    i32x4 q[RT][R::q_pieces];
    int lo[RT], hi[RT];
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

    f32x4 o[RT][DT];
    float mx[RT], sum[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      mx[rt] = kNegBig;
      sum[rt] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[rt][d] = f32x4{0, 0, 0, 0};
    }

    // the wave's tile t: its keys, their pages, their rows in the pool
    const int32_t *pages = c.table + (long long)s * c.max_pages;
    int page[NKH];
    auto load_pages = [&](int t) MOE_INLINE {
      const int k0 = range.key(t) + wave * C::keys;
#pragma unroll
      for (int kh = 0; kh < NKH; ++kh) {
        const int key = k0 + 16 * kh + l16;
        page[kh] = key < g.len ? pages[key >> c.page_shift] : -1;
      }
    };
    long long row[NKH];
    auto rows_of = [&](int t) MOE_INLINE {
      const int k0 = range.key(t) + wave * C::keys;
#pragma unroll
      for (int kh = 0; kh < NKH; ++kh) row[kh] = pool_row(c, page[kh], h, k0 + 16 * kh + l16);
    };
    i32x4 kr[NKH][R::pieces], vr[NKH][R::pieces];
    uint32_t ks[NKH][R::scales], vs[NKH][R::scales];
    auto load_rows = [&](const uint8_t *pool, const uint8_t *scale, i32x4 (&d)[NKH][R::pieces],
                         uint32_t (&sc)[NKH][R::scales]) MOE_INLINE {
#pragma unroll
      for (int kh = 0; kh < NKH; ++kh) {
        const long long r = row[kh] < 0 ? 0 : row[kh];
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
      for (int key = k0; key < k0 + C::keys && key < g.len; ++key) {
        const long long r = pool_row(c, pages[key >> c.page_shift], h, key);
        if (r < 0) continue;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const f32x4 v = not_finite4<F, HD>(c, r, 16 * d + 4 * g4);
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
    // tokens of the row tile
    const int tok_a = rt0 / a.group, tok_b = (min(rt0 + ROWS, nrows) - 1) / a.group;

    load_pages(t0);
    rows_of(t0);
    load_rows(c.k, c.k_scale, kr, ks);
    load_rows(c.v, c.v_scale, vr, vs);
    if (t0 + 1 < t1) load_pages(t0 + 1);

    for (int t = t0; t < t1; ++t) {
      const int k0 = range.key(t) + wave * C::keys;
      const bool more = t + 1 < t1;
      // keys that exist: bit l of half kh is key k0 + 16 kh + l
      uint32_t there[NKH];
      bool all = true;
#pragma unroll
      for (int kh = 0; kh < NKH; ++kh) {
        const unsigned long long m = __ballot(row[kh] >= 0);
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
      });
      __builtin_amdgcn_sched_barrier(0);
      if (more) {
        rows_of(t + 1);
        load_rows(c.k, c.k_scale, kr, ks);
      }
      __builtin_amdgcn_sched_barrier(0);

      // softmax over the tile; sc becomes the weights
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float top = mx[rt];
#pragma unroll
        for (int kh = 0; kh < NKH; ++kh)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 4 * g4 + i, key = k0 + 16 * kh + j;
            const bool see = ((there[kh] >> j) & 1) && key < hi[rt] && (key >= lo[rt] || key < a.sinks);
            const float v = see ? sc[rt][kh][i] * a.scale : -INFINITY;
            sc[rt][kh][i] = v;
            top = fmaxf(top, v);
          }
        top = max_rows16(top);
        const float alpha = __builtin_amdgcn_exp2f(mx[rt] - top);
        mx[rt] = top;
        float part = 0.0f;
#pragma unroll
        for (int kh = 0; kh < NKH; ++kh)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = __builtin_amdgcn_exp2f(sc[rt][kh][i] - top);
            sc[rt][kh][i] = p;
            part += p;
          }
        sum[rt] = sum[rt] * alpha + part;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[rt][d] *= alpha;
      }

      // V of keys that do not exist: zeros (their weight is zero, but zero times
      // what a free page holds need not be)
      if (!all)
        static_for<NKH>([&](auto kh) MOE_INLINE {
          if (row[kh] < 0) clear_v(vr[kh], vs[kh]);
        });
      // keys that some rows of the tile see and others do not
      bool unsafe = false;
      if (tok_b > tok_a && (k0 + C::keys > g.pos0 + tok_a + 1 || (a.window && k0 <= g.pos0 + tok_b - a.window)))
        static_for<NKH>([&](auto kh) MOE_INLINE { unsafe = unsafe || not_finite(vr[kh], vs[kh]); });
      const bool fix = __ballot(unsafe) != 0;
      if (fix) store_v(std::true_type{});
      else store_v(std::false_type{});
      __builtin_amdgcn_sched_barrier(0);
      if (more) {
        load_rows(c.v, c.v_scale, vr, vs);
        if (t + 2 < t1) load_pages(t + 2);
      }
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
    const bool whole = t0 == 0 && t1 == T;
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
    x += t1 - t0;
  }
}

// Join the pieces of cut units: a workgroup takes kJoinRows rows of a unit,
// 256 / (HD / 4) threads wide along the pieces.  It also clears the rows of
// no sequence.
constexpr int kJoinRows = 4;

template <int F, int HD, int RT, int NKH>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int units) {
  using C = RowsCfg<F, HD, RT, NKH>;
  constexpr int BK = C::BK, ROWS = C::rows, QUADS = ROWS / kJoinRows;
  constexpr int COLS = HD / 4, SL = 256 / COLS;    // columns of 4, slices of the pieces
  __shared__ f32x4 red[256];
  __shared__ float redm[SL][2];
  const KvArgs &c = a.c;
  const int tid = threadIdx.x, col = tid % COLS, sl = tid / COLS;
  clear_free_rows<F, HD>(a);
  const int quad = blockIdx.x % QUADS, h = blockIdx.x / QUADS % c.kv_heads;
  const int s = blockIdx.x / QUADS / c.kv_heads / units, rt = blockIdx.x / QUADS / c.kv_heads % units;
  const SeqGeo g = seq_geo(c, s);
  const int nrows = g.n * a.group, m0 = rt * ROWS + quad * kJoinRows;
  if (m0 >= nrows) return;
  const Cut<BK, ROWS> cut(a);
  const long long total = cut.total();
  const int runs = (int)min((long long)a.grid, total);
  const int T = Cut<BK, ROWS>::tiles(a, g);
  const long long x0 = cut.first(s) + (long long)(rt * c.kv_heads + h) * T, x1 = x0 + T;
  const int w0 = run_of(total, x0, runs), w1 = run_of(total, x1 - 1, runs);
  if (w0 == w1) return;                            // never cut: its workgroup wrote it
  const int first_slot = 2 * w0 + (run_start(total, w0, runs) == x0 ? 0 : 1);
  for (int mi = 0; mi < kJoinRows && m0 + mi < nrows; ++mi) {
    const int m = quad * kJoinRows + mi;
    float top = kNegBig, l = 0.0f;
    f32x4 acc = {0, 0, 0, 0};
    for (int w = w0 + sl; w <= w1; w += SL) {
      const float *p = a.part + (long long)(w == w0 ? first_slot : 2 * w) * ROWS * (HD + 2);
      const float pm = p[ROWS * HD + 2 * m], pl = p[ROWS * HD + 2 * m + 1];
      const f32x4 po = *(const f32x4 *)(p + m * HD + 4 * col);
      const float nt = fmaxf(top, pm);
      const float e0 = __builtin_amdgcn_exp2f(top - nt), e1 = __builtin_amdgcn_exp2f(pm - nt);
      acc = acc * e0 + po * e1;
      l = l * e0 + pl * e1;
      top = nt;
    }
    __syncthreads();
    red[tid] = acc;
    if (col == 0) { redm[sl][0] = top; redm[sl][1] = l; }
    __syncthreads();
    if (sl == 0) {
      float mt = kNegBig, lt = 0.0f;
      f32x4 at4 = {0, 0, 0, 0};
      for (int i = 0; i < SL; ++i) mt = fmaxf(mt, redm[i][0]);
      for (int i = 0; i < SL; ++i) {
        const float e = __builtin_amdgcn_exp2f(redm[i][0] - mt);
        lt += e * redm[i][1];
        at4 += e * red[i * COLS + col];
      }
      const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
      at4 *= inv;
      const int tok = (rt * ROWS + m) / a.group, hq = h * a.group + (rt * ROWS + m) % a.group;
      const long long at = ((long long)(g.r0 + tok) * a.heads + hq) * HD + 4 * col;
      if constexpr (F == FMT_F32)
        *(f32x4 *)((float *)a.out + at) = at4;
      else
        *(uint2 *)((uint16_t *)a.out + at) = make_uint2(bf16_pack2(at4[0], at4[1]), bf16_pack2(at4[2], at4[3]));
    }
  }
}

namespace {
constexpr int kRowsGrid = 512;                     // two workgroups a CU

template <int F, int HD, int RT, int NKH>
struct Launch {
  using C = RowsCfg<F, HD, RT, NKH>;
  static int units(const KvArgs &c, int group) {   // row tiles of the longest sequence
    return (int)(((long long)c.max_rows * group + C::rows - 1) / C::rows);
  }
  static int grid(const KvArgs &c, int group) {
    const long long tiles = (((long long)c.max_pages << c.page_shift) + C::BK - 1) / C::BK + 1;
    const long long all = (long long)c.seqs * c.kv_heads * units(c, group) * tiles;
    return (int)(all < kRowsGrid ? all : kRowsGrid);
  }
  static size_t ws(const KvArgs &c, int group) {
    return (size_t)grid(c, group) * 2 * C::rows * (HD + 2) * sizeof(float);
  }
  static hipError_t run(const AttnArgs &args, hipStream_t s) {
    AttnArgs a = args;
    a.grid = grid(a.c, a.group);
    static const hipError_t once = hipFuncSetAttribute(
        (const void *)attn_rows_kernel<F, HD, RT, NKH>, hipFuncAttributeMaxDynamicSharedMemorySize, C::lds);
    if (once != hipSuccess) return once;
    attn_rows_kernel<F, HD, RT, NKH><<<a.grid, 256, C::lds, s>>>(a);
    const int u = units(a.c, a.group);
    const long long joins = (long long)a.c.seqs * a.c.kv_heads * u * (C::rows / kJoinRows);
    if (joins > INT32_MAX) return hipErrorInvalidValue;
    attn_join_kernel<F, HD, RT, NKH><<<(unsigned)joins, 256, 0, s>>>(a, u);
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
  return pick(a.c, a.group, [&](auto l) { return l.ws(a.c, a.group); });
}
hipError_t launch_attn_rows(const AttnArgs &a, hipStream_t s) {
  return pick(a.c, a.group, [&](auto l) { return l.run(a, s); });
}

}  // namespace moe
