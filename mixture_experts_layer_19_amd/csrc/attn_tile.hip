// attn_tile.hip -- attention of chunks of new tokens over the paged cache.
//
// Bound by the matrix cores (bf16: 4 head_dim flops a row and key) and, next
// to them, by the exponentials and the LDS that feeds them.  A workgroup of
// NW waves takes 32 NW query rows (tokens x heads of the group) and walks the
// keys in tiles of 64; a wave owns 32 rows.  S^T = K Q^T and O^T = V^T P^T on
// 32x32 matrix instructions: a lane holds scores of one query only, so the
// running maximum and sum are per lane (one exchange between the half waves),
// rescaling needs no other lane, and the weights are already the operand that
// the second product reads.
//
// The loop is a pipeline over halves of a tile: while the softmax of one half
// runs on the vector units, the matrix cores work on the scores of the next
// and the values of the last (step, below).
//
// K and V tiles come through registers (MX codes become bf16 there, exactly)
// into two LDS buffers each, with one barrier a tile.  Rows are longer than
// their data, so that the reads, K's by rows and V's transposed, spread over the
// banks (TileCfg), and every read's address is one register and a constant.
//
// The running maximum is a reference that moves only when a score passes it
// by 2^8: the weights stay below 2^8 of fp32 and the output is rescaled rarely.
//
// Few units: each is cut into `splits` runs of tiles, joined from the
// workspace in the order of their keys (attn_tile_join_kernel).
//
// Measured, 64 heads over 8 KV heads of 128: 4 chunks of 640-1408 tokens over up
// to 7501 bf16 keys before them 866 us (994 TFLOP/s; the matrix cores work 49% of
// the time, the vector units 45%), 4001 tokens under a window of 1024 over
// MX-fp8 209 us (645).  The same chunks at head_dim 64 545 us (789), 256 2440 (705).
#include "attn_common.hpp"

namespace moe {

template <int F, int HD, int NW>
struct TileCfg {
  static constexpr int threads = 64 * NW, rows = 32 * NW;  // query rows of a workgroup
  static constexpr int BK = 64;                            // keys of a tile
  static constexpr int elem = F == FMT_F32 ? 4 : 2;        // in LDS
  static constexpr int row_bytes = HD * elem, chunks = row_bytes / 16;
  // Rows in LDS.  Of K, 16 lanes read 16 bytes each of 16 rows: 4 banks further a
  // row.  Of V, 32 lanes read 64 bytes each of 4 rows: 16 banks further a row (no
  // conflicts counted).  fp32 reads 128 bytes each of 2 rows of V that share
  // their banks: 84 us for the mixed batch, and 90 with rows 32 bytes longer.
  static constexpr int k_pitch = row_bytes + 16, v_pitch = row_bytes + (F == FMT_F32 ? 0 : 64);
  static constexpr int k_tile = BK * k_pitch, v_tile = BK * v_pitch;
  static constexpr int lds = 2 * (k_tile + v_tile) + 8 * NW;
  // staging of K or V, pieces of 16 bytes a thread: bf16 and fp32 by chunk, MX
  // 16 codes or more of one key (parts threads a key; threads beyond them do
  // what others do)
  static constexpr int parts = HD / 16 < NW ? HD / 16 : NW, codes = HD / parts, scales = codes > 32 ? codes / 32 : 1;
  static constexpr int pieces = F == FMT_MX8 ? codes / 16 : BK * row_bytes / 16 / threads;
  static constexpr int span = F == FMT_MX8 ? 1 : 64 / chunks;   // keys of a wave's piece (of one page)
  static constexpr int QP = row_bytes / 32;                // 16-byte query pieces a lane
  static constexpr int DT = HD / 32;
};

// Sequence and row tile of unit u, or s = -1 past the last unit.  Long units
// come first, so that the last ones to start are short: of each 64 sequences
// the longest first, the row tiles of a sequence from its end.
template <int ROWS>
__device__ __forceinline__ void find_unit(const AttnArgs &a, int u, int &s, int &rt) {
  const int lane = threadIdx.x & 63;
  s = -1;
  rt = 0;
  for (int s0 = 0; s0 < a.c.seqs; s0 += 64) {
    int units = 0, len = -1;
    if (s0 + lane < a.c.seqs) {
      const SeqGeo g = seq_geo(a.c, s0 + lane);
      units = (int)(((long long)g.n * a.group + ROWS - 1) / ROWS);
      len = g.len;
    }
    const int n = min(a.c.seqs - s0, 64);
    int rank = 0;                                  // sequences before this one
    for (int i = 0; i < n; ++i) {
      const int other = __builtin_amdgcn_readlane(len, i);
      rank += other > len || (other == len && i < lane);
    }
    if (lane >= n) rank = lane;
    // lane r: the sequence of rank r
    const int seq = __builtin_amdgcn_ds_permute(rank << 2, lane);
    const int v = wave_scan(__shfl(units, seq, 64));
    const unsigned long long past = __ballot(v > u);
    if (past) {
      const int l = __ffsll((long long)past) - 1;
      s = s0 + __builtin_amdgcn_readlane(seq, l);
      rt = __builtin_amdgcn_readlane(v, l) - 1 - u;               // descending
      return;
    }
    u -= __builtin_amdgcn_readlane(v, 63);
  }
}

template <int F, int HD, int NW, int OCC>
__global__ __launch_bounds__(64 * NW, OCC) void attn_tile_kernel(AttnArgs a, int splits) {
  using C = TileCfg<F, HD, NW>;
  constexpr int ROWS = C::rows, BK = C::BK, DT = C::DT, QP = C::QP, NP = C::pieces;
  constexpr int KEYS = F == FMT_MX8 ? 1 : NP;              // places that a thread stages pieces from
  extern __shared__ __align__(16) uint8_t lds[];           // K0 K1 V0 V1, flags
  int *flags = (int *)(lds + 2 * (C::k_tile + C::v_tile));   // [stage][wave]
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

  // query: lane q32 holds row m
  i32x4 q[QP];
  const int m0 = rt0 + 32 * wave, m = m0 + q32;
  const bool in = m < nrows, has_rows = m0 < nrows;
  const int own_tok = in ? m / a.group : 0, hq = h * a.group + (in ? m % a.group : 0);
  {
    const uint8_t *qp =
        (const uint8_t *)a.q + ((long long)(g.r0 + own_tok) * a.q_row + hq * a.q_head) * C::elem + 16 * hf;
#pragma unroll
    for (int p = 0; p < QP; ++p) q[p] = in ? *(const i32x4 *)(qp + 32 * p) ^ (int)a.q_sign : i32x4{0, 0, 0, 0};
  }
  const RowMask mask(g, own_tok, in, a.window, a.sinks);
  // keys that all rows of the workgroup see (but for the sinks)
  const int all_hi = min(g.pos0 + tok_a + 1, g.len), all_lo = a.window ? g.pos0 + tok_b - a.window + 1 : 0;

  f32x16 o[DT];
  float mx = kNegBig, sum = 0.0f;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;

  // ---- staging
  const int32_t *pages = c.table + (long long)s * c.max_pages;
  // key of the tile that piece p of this thread belongs to (MX: all pieces)
  auto piece_key = [&](int p) MOE_INLINE {
    if constexpr (F == FMT_MX8) return tid / C::parts % BK;
    else return (p * C::threads + tid) / C::chunks;
  };
  // The table's entry for key `lane` of tile t (MX: and for the thread's piece),
  // and the rows of the pool there.  A bf16 or fp32 piece of a wave is `span`
  // consecutive keys, all in one page (pages hold 8 keys or more), so its row is
  // a scalar, taken from the lane that looked it up, and its lanes read a
  // contiguous KiB.  As in the row kernel no load of the loop stands under a
  // condition: past the last tile, and for keys without a page, row 0 is read.
  struct Pages {
    int lane, piece;
  };
  auto pages_of = [&](int t) MOE_INLINE {
    const int k0 = range.key(min(t, t1 - 1));
    Pages r;
    r.lane = pages[min((k0 + lane) >> c.page_shift, c.max_pages - 1)];
    r.piece = F == FMT_MX8 ? pages[min((k0 + piece_key(0)) >> c.page_shift, c.max_pages - 1)] : 0;
    return r;
  };
  struct Rows {
    uint32_t piece[KEYS];
    unsigned long long have;                               // bit j: key j of the tile exists
  };
  auto rows_of = [&](int t, const Pages &page) MOE_INLINE {
    const int k0 = range.key(t), left = t < t1 ? g.len - k0 : 0;
    const bool in = (unsigned)page.lane < (unsigned)c.num_pages && lane < left;
    Rows r;
    r.have = __ballot(in);
    if constexpr (F == FMT_MX8) {
      const uint32_t row = pool_row(c, page.piece, h, k0 + piece_key(0));
      r.piece[0] = row != kNoRow && piece_key(0) < left ? row : 0u;
    } else {
      const uint32_t row = in ? pool_row(c, page.lane, h, k0 + lane) : 0u;
#pragma unroll
      for (int p = 0; p < KEYS; ++p) r.piece[p] = __builtin_amdgcn_readlane(row, (p * NW + wave) * C::span);
    }
    return r;
  };
  // a tile's K or V on its way
  struct Stage {
    i32x4 d[NP];
    uint32_t scale[C::scales];
  };
  auto load_tile = [&](Stage &st, const uint8_t *pool, const uint8_t *scale, const Rows &r) MOE_INLINE {
    if constexpr (F == FMT_MX8) {
      const long long at = (long long)r.piece[0] * HD + tid % C::parts * C::codes;
#pragma unroll
      for (int p = 0; p < NP; ++p) st.d[p] = *(const i32x4 *)(pool + at + 16 * p);
#pragma unroll
      for (int i = 0; i < C::scales; ++i) st.scale[i] = scale[(at >> 5) + i];
    } else {
#pragma unroll
      for (int p = 0; p < NP; ++p)
        st.d[p] = *(const i32x4 *)(pool + (unsigned long long)r.piece[p] * C::row_bytes + 16u * lane);
    }
  };
  // (`finite`: zeros in place of what is not)
  auto put = [&](const Stage &st, uint8_t *tile, int pitch, auto finite) MOE_INLINE {
    auto chunk = [&](int key, int ch, uint4 w) MOE_INLINE {
      if constexpr (finite)
        w = make_uint4(word_finite<F>(w.x), word_finite<F>(w.y), word_finite<F>(w.z), word_finite<F>(w.w));
      *(uint4 *)(tile + key * pitch + (ch << 4)) = w;
    };
    if constexpr (F == FMT_MX8) {
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t sb = st.scale[p * 16 / 32 % C::scales];
          const uint2 w0 = e4m3_to_bf16x4(st.d[p][2 * x], sb), w1 = e4m3_to_bf16x4(st.d[p][2 * x + 1], sb);
          chunk(piece_key(0), tid % C::parts * (C::codes / 8) + 2 * p + x, make_uint4(w0.x, w0.y, w1.x, w1.y));
        }
    } else {
#pragma unroll
      for (int p = 0; p < NP; ++p) chunk(piece_key(p), (p * C::threads + tid) % C::chunks, __builtin_bit_cast(uint4, st.d[p]));
    }
  };
  // Tiles whose keys all exist and are seen by all rows: no masks, and no need
  // to look for values that are not finite.
  auto plain = [&](int t, unsigned long long have) MOE_INLINE {
    const int k0 = range.key(t);
    return k0 + BK <= all_hi && k0 >= all_lo && have == ~0ull;
  };
  auto k_tile = [&](int t) MOE_INLINE { return lds + ((t - t0) & 1) * C::k_tile; };
  auto v_tile = [&](int t) MOE_INLINE { return lds + 2 * C::k_tile + ((t - t0) & 1) * C::v_tile; };
  auto store_v = [&](Stage &st, int t, unsigned long long have) MOE_INLINE {
    if (have != ~0ull) {                                   // V of keys that do not exist: zeros
#pragma unroll
      for (int p = 0; p < NP; ++p)
        if (!((have >> piece_key(p)) & 1)) {
          st.d[p] = i32x4{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < C::scales; ++i) st.scale[i] = 0;
        }
    }
    if (!plain(t, have)) {
      put(st, v_tile(t), C::v_pitch, std::true_type{});
      bool bad = false;
      if constexpr (F == FMT_MX8)
#pragma unroll
        for (int i = 0; i < C::scales; ++i) bad = bad || st.scale[i] >= kScaleOverflow;
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) bad = bad || word_not_finite<F>((uint32_t)st.d[p][i]);
      const unsigned long long any = __ballot(bad);
      if (lane == 0) flags[NW * ((t - t0) & 1) + wave] = any != 0;
    } else {
      put(st, v_tile(t), C::v_pitch, std::false_type{});
    }
  };

  // ---- products, of halves of a tile (32 keys).  Addresses within LDS of the
  // lane's first reads; the first V buffer that is read is that of the tile
  // before the first.
  const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t *)lds;
  uint32_t k_addr = lds0 + q32 * C::k_pitch + 16 * hf;
  uint32_t v_addr = lds0 + 2 * C::k_tile + C::v_tile +
                    (F == FMT_F32 ? 4 * hf * C::v_pitch + 4 * q32
                                  : (4 * hf + ((lane & 15) >> 2)) * C::v_pitch + 32 * ((lane >> 4) & 1) + 8 * (lane & 3));
  const uint32_t k_both = 2 * k_addr + C::k_tile, v_both = 2 * v_addr - C::v_tile;
  auto other_buffers = [&]() MOE_INLINE {
    k_addr = k_both - k_addr;
    v_addr = v_both - v_addr;
  };
  // The products of a step, in slots: even ones a piece of the scores' head_dim
  // (S^T; element i is key 8 (i / 4) + 4 hf + i % 4 of the half), odd ones 16
  // keys (fp32: 4) of the values for 32 columns.  So neighbours do not wait for
  // each other's sums.
  constexpr int PV = F == FMT_F32 ? 4 : 2, SLOTS = QP + PV * DT;
  static_assert(QP == PV * DT, "as many pieces of scores as of values");
  // the softmax weights of a half: fp32, or bf16 in pairs
  using Weights = std::conditional_t<F == FMT_F32, f32x16, i32x8>;
  auto read_k = [&](auto n, int half) MOE_INLINE {
    using P = const __attribute__((address_space(3))) i32x4 *;
    return *(P)(size_t)(k_addr + 32 * half * C::k_pitch + 32 * n);
  };
  auto read_v = [&](auto n, int half) MOE_INLINE {
    constexpr int dt = n % DT, part = n / DT;
    i32x4 f;
    if constexpr (F == FMT_F32) {
      using P = const __attribute__((address_space(3))) int *;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = *(P)(size_t)(v_addr + (32 * half + 8 * part + i) * C::v_pitch + 128 * dt);
    } else {
      // a group of 16 lanes reads 4 keys x 16 columns, transposed
      using P = __attribute__((address_space(3))) s16x4 *;
      const i32x2 v0 = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (P)(size_t)(v_addr + (32 * half + 16 * part) * C::v_pitch + 64 * dt)));
      const i32x2 v1 = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (P)(size_t)(v_addr + (32 * half + 16 * part + 8) * C::v_pitch + 64 * dt)));
      f = __builtin_shufflevector(v0, v1, 0, 1, 2, 3);
    }
    return f;
  };
  auto mul_k = [&](f32x16 &sc, const i32x4 &k, auto n) MOE_INLINE {
    if constexpr (F == FMT_F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sc = __builtin_amdgcn_mfma_f32_32x32x2f32(__int_as_float(k[e]), __int_as_float(q[n][e]), sc, 0, 0, 0);
    } else {
      sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, k), __builtin_bit_cast(bf16x8, q[n]), sc,
                                                   0, 0, 0);
    }
  };
  auto mul_v = [&](const Weights &w, const i32x4 &v, auto n) MOE_INLINE {
    constexpr int dt = n % DT, part = n / DT;
    if constexpr (F == FMT_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[dt] = __builtin_amdgcn_mfma_f32_32x32x2f32(__int_as_float(v[i]), w[4 * part + i], o[dt], 0, 0, 0);
    } else {
      const i32x4 pw = {w[4 * part], w[4 * part + 1], w[4 * part + 2], w[4 * part + 3]};
      o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, pw),
                                                     o[dt], 0, 0, 0);
    }
  };
  // what is not finite of V in half `half` of a tile that is not plain (zeros
  // in LDS)
  auto add_not_finite = [&](int t, int half) MOE_INLINE {
    const int *f = flags + NW * ((t - t0) & 1);
    int any = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) any |= f[i];
    if (!any) return;
    int d0 = 4 * hf;
    asm volatile("" : "+v"(d0));                   // its addresses stay out of the loop's registers
    const int k0 = range.key(t) + 32 * half;
    for (int key = k0; key < k0 + 32 && key < g.len; ++key) {
      const uint32_t r = pool_row(c, pages[key >> c.page_shift], h, key);
      if (r == kNoRow) continue;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const f32x4 v = not_finite4<F, HD>(c, r, 32 * d + 8 * b + d0);
          if (mask.sees(key))
#pragma unroll
            for (int i = 0; i < 4; ++i) o[d][4 * b + i] += v[i];
        }
    }
  };
  // One half: cur holds its scores and becomes the weights w; meanwhile the
  // next half's scores go to next, and the last half's weights last multiply
  // its values.  The three do not depend on each other, so the matrix cores run
  // under the softmax of the same wave.
  //   half 0: next = half 1 of tile t, last = half 1 of tile t - 1
  //   half 1: next = half 0 of tile t + 1, last = half 0 of tile t
  // begin issues the first reads; what stands between it and step runs under them.
  constexpr int AHEAD = 2;                         // slots between a read and its product
  i32x4 frag[AHEAD];
  auto read = [&](auto half, auto n) MOE_INLINE {
    if constexpr (n % 2) frag[n % AHEAD] = read_v(std::integral_constant<int, n / 2>{}, 1 - half);
    else frag[n % AHEAD] = read_k(std::integral_constant<int, n / 2>{}, 1 - half);
  };
  auto begin = [&](auto half) MOE_INLINE {
    static_for<AHEAD>([&](auto n) MOE_INLINE { read(half, n); });
    __builtin_amdgcn_sched_barrier(0);
  };
  const int far_exp = far_exponent(a.scale);
  auto step = [&](auto half, int t, unsigned long long have, bool is_plain, bool v_plain, f32x16 &cur, f32x16 &next,
                  Weights &w, const Weights &last) MOE_INLINE {
    if (!is_plain) {
      const int k0 = range.key(t) + 32 * half;
      uint32_t bits = (uint32_t)(have >> (32 * half)) >> (4 * hf);
      asm volatile("" : "+v"(bits));               // keeps the masks out of plain tiles
      const int base = k0 + 4 * hf, below = mask.hi - base, from = mask.lo - base, sink = a.sinks - base;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = 8 * (i / 4) + i % 4;
        const bool see = ((bits >> j) & 1) && j < below && (j >= from || j < sink);
        cur[i] = see ? cur[i] : -INFINITY;
      }
    }
    // The slots in this order.  The maximum comes first, the exponentials are
    // spread over the slots, and their sum and rounding follow one slot behind.
    constexpr int FIRST = 2, SPAN = SLOTS - FIRST - 1;
    __builtin_amdgcn_sched_barrier(0);
    bool far = false;
    float top = -INFINITY, now = 0.0f, alpha = 0.0f, mul = a.scale, part[2] = {0.0f, 0.0f};
    static_for<SLOTS>([&](auto n) MOE_INLINE {
      if constexpr (n == 0)
#pragma unroll
        for (int i = 0; i < 16; ++i) next[i] = 0.0f;
      if constexpr (n % 2) mul_v(last, frag[n % AHEAD], std::integral_constant<int, n / 2>{});
      else mul_k(next, frag[n % AHEAD], std::integral_constant<int, n / 2>{});
      if constexpr (n + AHEAD < SLOTS) read(half, std::integral_constant<int, n + AHEAD>{});
      if constexpr (n == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, cur[i]);
        far = __ballot(__builtin_amdgcn_frexp_expf(top) > far_exp) != 0;
      }
      if constexpr (n == 1) {
        top = max_half(top) * a.scale;             // the scale is positive
        // the reference moves only when a score passes it by 2^8
        now = top > mx + 8.0f ? top : mx;
        alpha = __builtin_amdgcn_exp2f(mx - now);
        if (__builtin_expect(far, 0)) {
          asm volatile("");                        // a branch, not selects
          mul = 1.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) cur[i] *= a.scale;
        }
      }
      // elements whose exponentials are due in slot n: [due(n), due(n + 1))
      auto due = [](int m) constexpr { return m <= FIRST ? 0 : m >= FIRST + SPAN ? 16 : 16 * (m - FIRST) / SPAN; };
      constexpr int e0 = due(n), e1 = due(n + 1), d0 = due(n - 1);
#pragma unroll
      for (int i = e0; i < e1; ++i) cur[i] = __builtin_amdgcn_exp2f(fmaf(cur[i], mul, -now));
#pragma unroll
      for (int i = d0; i < e0; ++i) {
        part[i % 2] += cur[i];
        if constexpr (F != FMT_F32)
          if (i % 2) w[i / 2] = (int)bf16_pack2(cur[i - 1], cur[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (F == FMT_F32) w = cur;
    sum = fmaf(sum, alpha, part[0] + part[1]);
    asm volatile("" : "+v"(w), "+v"(sum));         // ahead of the branches below
    if (!v_plain) add_not_finite(half ? t : t - 1, 1 - half);
    const bool moved = now > mx;
    mx = now;
    if (__ballot(moved)) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
    }
  };

  if (t0 < t1) {
    // Ahead of the loop: K of two tiles, V of one, zeros for the values of the
    // half before the first (whose weights are zero).  In iteration t: K of
    // t + 2 and V of t + 1 come in; the one barrier stands between the last
    // reads of the buffers that they go to and the stores.
    constexpr std::integral_constant<int, 0> first{};
    constexpr std::integral_constant<int, 1> second{};
    Rows row = rows_of(t0, pages_of(t0)), row1 = rows_of(t0 + 1, pages_of(t0 + 1));
    Stage sk, sv;
    {
      Stage s0;
      load_tile(s0, c.k, c.k_scale, row);
      load_tile(sv, c.v, c.v_scale, row);
      load_tile(sk, c.k, c.k_scale, row1);
      put(s0, k_tile(t0), C::k_pitch, std::false_type{});
      store_v(sv, t0, row.have);
      put(sk, k_tile(t0 + 1), C::k_pitch, std::false_type{});
    }
    Pages page = pages_of(t0 + 2);
    for (int i = tid; i < 32 * C::v_pitch / 16; i += C::threads)
      *(uint4 *)(v_tile(t0 + 1) + 32 * C::v_pitch + 16 * i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    f32x16 sa, sb;
    Weights wa, wb;
#pragma unroll
    for (int i = 0; i < (F == FMT_F32 ? 16 : 8); ++i) wb[i] = 0;
    if (has_rows) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sa[i] = 0.0f;
      static_for<QP>([&](auto n) MOE_INLINE { mul_k(sa, read_k(n, 0), n); });
    }
    bool is_plain = plain(t0, row.have), last_plain = true;
    for (int t = t0; t < t1; ++t) {
      if (has_rows) begin(first);
      const Rows row2 = rows_of(t + 2, page);
      load_tile(sk, c.k, c.k_scale, row2);
      load_tile(sv, c.v, c.v_scale, row1);
      page = pages_of(t + 3);
      if (has_rows) step(first, t, row.have, is_plain, last_plain, sa, sb, wa, wb);
      other_buffers();
      // The barrier, without waiting for the loads: LDS accesses are done.
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (has_rows) {
        begin(second);
        step(second, t, row.have, is_plain, is_plain, sb, sa, wb, wa);
      }
      row = row1;
      row1 = row2;
      put(sk, k_tile(t + 2), C::k_pitch, std::false_type{});
      last_plain = is_plain;
      if (t + 1 < t1) {
        is_plain = plain(t + 1, row.have);
        store_v(sv, t + 1, row.have);
      }
    }
    if (has_rows) {
      static_for<PV * DT>([&](auto n) MOE_INLINE { mul_v(wb, read_v(n, 1), n); });
      if (!last_plain) add_not_finite(t1 - 1, 1);
    }
  }

  // ---- results
  const float l = sum_half(sum);
  if (in) {
    if (splits == 1) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const long long at = ((long long)(g.r0 + own_tok) * a.heads + hq) * HD + 4 * hf;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float v0 = o[d][4 * b] * inv, v1 = o[d][4 * b + 1] * inv;
          const float v2 = o[d][4 * b + 2] * inv, v3 = o[d][4 * b + 3] * inv;
          if constexpr (F == FMT_F32)
            *(f32x4 *)((float *)a.out + at + 32 * d + 8 * b) = f32x4{v0, v1, v2, v3};
          else
            *(uint2 *)((uint16_t *)a.out + at + 32 * d + 8 * b) = make_uint2(bf16_pack2(v0, v1), bf16_pack2(v2, v3));
        }
    } else {
      float *part = a.part + (((long long)u * c.kv_heads + h) * splits + split) * ROWS * (HD + 2);
      const int r = m - rt0;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *(f32x4 *)(part + r * HD + 32 * d + 8 * b + 4 * hf) =
              f32x4{o[d][4 * b], o[d][4 * b + 1], o[d][4 * b + 2], o[d][4 * b + 3]};
      if (hf == 0) {
        part[ROWS * HD + 2 * r] = mx;
        part[ROWS * HD + 2 * r + 1] = l;
      }
    }
  }
  clear_free_rows<F, HD>(a);
}

// Join the splits of a unit: HD / 4 threads a row, 4 columns each.
template <int F, int HD, int NW>
__global__ __launch_bounds__(256) void attn_tile_join_kernel(AttnArgs a, int splits) {
  constexpr int ROWS = TileCfg<F, HD, NW>::rows, COLS = HD / 4, PER = 256 / COLS;
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
template <int F, int HD, int NW, int OCC>
struct TileLaunch {
  using C = TileCfg<F, HD, NW>;
  // row tiles of all sequences, at most
  static long long units(const AttnArgs &a) {
    const long long each = ((long long)a.c.max_rows * a.group + C::rows - 1) / C::rows * a.c.seqs;
    const long long all = (long long)a.c.rows * a.group / C::rows + a.c.seqs;
    return each < all ? each : all;
  }
  // Enough workgroups for every CU (OCC of four waves), but four
  // key tiles at least in a run where the longest possible row sees that many.
  // fp32 of head_dim 64 is bound by its slow matrix instructions and by uneven
  // units: twice as many (12 sequences of 1-211 tokens over up to 900 keys, 16
  // heads: 110 -> 87 us; four times: 103; bf16 and larger heads lose).
  static int splits(const AttnArgs &a) {
    const long long wgs = units(a) * a.c.kv_heads, want = 256 * OCC * 4 / NW * (F == FMT_F32 && HD == 64 ? 2 : 1);
    long long keys = (long long)a.c.max_pages << a.c.page_shift;
    if (a.window) {
      const long long seen = (long long)a.window + a.sinks + C::rows / a.group + 1;
      keys = keys < seen ? keys : seen;
    }
    const long long most = keys / (4 * C::BK) < 1 ? 1 : keys / (4 * C::BK);
    const long long s = want / wgs;
    return (int)(s < 1 ? 1 : s < most ? s : most);
  }
  static bool fits(const AttnArgs &a) {
    const long long u = units(a) * a.c.kv_heads;
    return u * splits(a) <= max_groups(C::threads) && u * (C::rows / (1024 / HD)) <= max_groups(256);
  }
  static size_t ws(const AttnArgs &a) {
    const int s = splits(a);
    return s == 1 ? 0 : (size_t)units(a) * a.c.kv_heads * s * C::rows * (HD + 2) * sizeof(float);
  }
  static hipError_t run(const AttnArgs &a, hipStream_t st) {
    const int s = splits(a);
    const long long u = units(a) * a.c.kv_heads, grid = u * s;
    static OncePerDevice once;
    const hipError_t err = allow_lds(once, (const void *)attn_tile_kernel<F, HD, NW, OCC>, C::lds);
    if (err != hipSuccess) return err;
    attn_tile_kernel<F, HD, NW, OCC><<<(unsigned)grid, C::threads, C::lds, st>>>(a, s);
    if (s > 1)
      attn_tile_join_kernel<F, HD, NW><<<(unsigned)(u * (C::rows / (1024 / HD))), 256, 0, st>>>(a, s);
    return hipGetLastError();
  }
};

// Waves a workgroup and workgroups of four waves a CU: as many as the registers
// hold.  head_dim 64 at three (bf16 8 registers short, kept in memory) against
// two: chunks of 640-1408 tokens over up to 7501 keys 562 and 598 us, a window
// of 1024 129 and 147; one of eight waves: 606.  head_dim 256 fills a wave's
// registers (bf16 keeps 36 bytes a lane in memory).
template <typename Fn>
auto pick_tile(const KvArgs &c, Fn &&f) {
  if (c.fmt == FMT_F32) return c.head_dim == 64 ? f(TileLaunch<FMT_F32, 64, 4, 2>{}) : f(TileLaunch<FMT_F32, 128, 4, 1>{});
  if (c.fmt == FMT_BF16) {
    if (c.head_dim == 64) return f(TileLaunch<FMT_BF16, 64, 4, 3>{});
    if (c.head_dim == 128) return f(TileLaunch<FMT_BF16, 128, 8, 2>{});
    return f(TileLaunch<FMT_BF16, 256, 4, 1>{});
  }
  if (c.head_dim == 64) return f(TileLaunch<FMT_MX8, 64, 4, 3>{});
  if (c.head_dim == 128) return f(TileLaunch<FMT_MX8, 128, 8, 2>{});
  return f(TileLaunch<FMT_MX8, 256, 4, 1>{});
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
