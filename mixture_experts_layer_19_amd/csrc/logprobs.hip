// logprobs.hip -- log probabilities of given tokens, the entropy, and the best
// alternatives of each row of logits.
//
//   log p(t) = x_t - m - log l,       m = max x,  l = sum e^(x - m)
//   H        = log l - sum (x - m) e^(x - m) / l
//   top:       the n best (value, then lower index) with their log probabilities
//
// One pass: a thread keeps a running maximum with the two sums under it (exponents in
// units of log 2; fp32) over vectors of 16 bytes, four of bf16 at once; the threads'
// sums are joined in a fixed order.  The alternatives need no second pass over the row:
// at least n elements are not below the n-th largest of the threads' maxima, so the
// n best lie in the vectors of the few threads whose maximum is not below it either, and
// only those are read again (from the L2).  What is not below it there, some n elements
// and ties, goes into a list in LDS; each takes its place by counting the larger ones.
// Elements compare as 64-bit keys, the value's order above the index's complement, so
// that there are no ties, and the list's own order does not matter.  Where fewer groups
// of threads than n hold a finite logit, every thread is such a one: the row is read
// again as a whole and the list cut down as it goes (64 rows of 120832 fp32, 20 alternatives:
// 54 us with 5 or 20 tokens not masked, 16 with 300 and more).
//
// Bound by memory where rows are many (4096 of 120832 bf16: 181 us, 5.5 TB/s; 2048 of
// 32003, which are not 16-byte aligned: 33.5 us, 3.9 TB/s); a row by itself is read by one
// workgroup, which one CU's share of the bandwidth and the steps behind the pass bound (one of
// 120832 fp32: 11.5 us, with 5 alternatives 14.0, with 64 16.7).
#include "block_common.hpp"

namespace moe {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
constexpr int kList = 512;                       // keys that are ranked by counting
static_assert(kLogprobTop <= 64 && kLogprobTop <= kList, "n-th largest of the maxima");

// Order of a value as an unsigned number: NaN 0, then -infinity upwards; -0 is 0.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return v != v ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return o == 0 ? __builtin_nanf("") : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t i) { return (uint64_t)order_of(v) << 32 | (0xFFFFFFFFu - i); }

// l = sum e^(x - m), t = sum (x - m) / ln 2 e^(x - m) of some elements; none: l = 0.
struct Sums {
  float m, l, t;
};
// The distance of two maxima in units of log 2, for factors e^: what is infinitely
// far (or NaN, of two infinities) goes to a finite one with the factor 0.
__device__ __forceinline__ float apart(float from, float to) { return fmaxf((from - to) * kLog2e, -1.0e4f); }
// (no fused operations: either order of the two gives the same bits, and so every thread
// that joins the same sums)
__device__ __forceinline__ Sums join(const Sums &a, const Sums &b) {
#pragma clang fp contract(off)
  Sums r;
  r.m = fmaxf(a.m, b.m);
  const float da = apart(a.m, r.m), db = apart(b.m, r.m);
  const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
  r.l = a.l * fa + b.l * fb;
  r.t = (a.t + a.l * da) * fa + (b.t + b.l * db) * fb;
  return r;
}
template <int N>
__device__ __forceinline__ void add(Sums &s, const float (&v)[N]) {
  float top = v[0];
#pragma unroll
  for (int j = 1; j < N; ++j) top = fmaxf(top, v[j]);
  if (top > s.m) {
    const float d = apart(s.m, top), f = __builtin_amdgcn_exp2f(d);
    s.t = fmaf(s.l, d, s.t) * f;
    s.l *= f;
    s.m = top;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float d = (v[j] - s.m) * kLog2e, e = __builtin_amdgcn_exp2f(d);
    s.l += e;
    s.t = fmaf(e, fmaxf(d, -200.0f), s.t);       // e is 0 there; 0 x -infinity would be NaN
  }
}
// T threads a row; vectors of E elements.
template <int T, int E>
struct __align__(16) LogprobLds {
  static constexpr int waves = T / 64, keys = kList + T * E, per = (keys + T - 1) / T;
  static constexpr int groups = T < 256 ? T : 256;         // of threads, whose maxima are ordered
  uint64_t list[keys];           // what one sweep of all threads may add beyond those that are ranked
  uint32_t most[groups];         // order of the maximum of each group of threads
  uint32_t owner[T];
  Sums red[waves];
  int owners, count, tally[2];
  uint32_t least;
};
// The sums of all threads, in every thread.
template <int WAVES>
__device__ __forceinline__ Sums join_group(Sums s, Sums *red) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1)
    s = join(s, Sums{__shfl_xor(s.m, m, 64), __shfl_xor(s.l, m, 64), __shfl_xor(s.t, m, 64)});
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  s = red[threadIdx.x % WAVES];
#pragma unroll
  for (int m = 1; m < WAVES; m <<= 1)
    s = join(s, Sums{__shfl_xor(s.m, m, 64), __shfl_xor(s.l, m, 64), __shfl_xor(s.t, m, 64)});
  return s;
}

// The n-th largest of the list's `count` keys (n <= count; keys differ): bit by bit.
template <int T, int E>
__device__ __forceinline__ uint64_t nth_largest(LogprobLds<T, E> &s, int count, int n) {
  constexpr int PER = LogprobLds<T, E>::per;
  uint64_t k[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) k[i] = i * T + (int)threadIdx.x < count ? s.list[i * T + threadIdx.x] : 0;
  uint64_t found = 0;
  if (threadIdx.x < 2) s.tally[threadIdx.x] = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t trial = found | 1ull << bit;
    int c = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c += __popcll(__ballot(k[i] >= trial));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) atomicAdd(&s.tally[bit & 1], c);
    __syncthreads();
    if (s.tally[bit & 1] >= n) found = trial;
    if (threadIdx.x == 0) s.tally[~bit & 1] = 0;
  }
  return found;
}
// Leave the list's n largest keys in it (n <= count); the smallest of them.
template <int T, int E>
__device__ __forceinline__ uint64_t prune(LogprobLds<T, E> &s, int count, int n) {
  constexpr int PER = LogprobLds<T, E>::per;
  const uint64_t least = nth_largest(s, count, n);
  uint64_t k[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) k[i] = i * T + (int)threadIdx.x < count ? s.list[i * T + threadIdx.x] : 0;
  __syncthreads();
  if (threadIdx.x == 0) s.count = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (k[i] >= least) s.list[atomicAdd(&s.count, 1)] = k[i];
  __syncthreads();
  return least;
}
__device__ __forceinline__ void write_row(const LogprobArgs &a, int row, const Sums &s) {
  const long long token = a.token_bytes == 8 ? ((const long long *)a.tokens)[row] : ((const int32_t *)a.tokens)[row];
  float x = -INFINITY;
  if (token >= 0 && token < a.vocab) {
    const long long at = (long long)row * a.stride + token;
    x = a.is_bf16 ? bf16_to_f32(((const uint16_t *)a.logits)[at]) : ((const float *)a.logits)[at];
  }
  float lp = x - s.m - logf(s.l), h = kLn2 * (__log2f(s.l) - s.t / s.l);
  if (s.l == 0.0f || (x == -INFINITY && s.l == s.l)) lp = -INFINITY;       // nothing, or not this token, has a probability
  if (s.l == 0.0f || h < 0.0f) h = 0.0f;
  a.logprob[row] = lp;
  a.entropy[row] = h;
}
__device__ __forceinline__ void write_top(const LogprobArgs &a, int row, const Sums &s, int place, uint64_t key) {
  const float x = value_of((uint32_t)(key >> 32));
  const long long at = (long long)row * a.top + place;
  a.top_logprob[at] = s.l == 0.0f || (x == -INFINITY && s.l == s.l) ? -INFINITY : x - s.m - logf(s.l);
  a.top_token[at] = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
}

// A row a workgroup of T threads.
template <bool BF16, int T>
__global__ __launch_bounds__(T) void logprob_kernel(LogprobArgs a, int first) {
  constexpr int E = BF16 ? 8 : 4, U = BF16 ? 4 : 8;        // elements of a vector, vectors at once
  __shared__ LogprobLds<T, E> s;
  const int tid = threadIdx.x, row = first + (int)blockIdx.x;
  const uint8_t *x = (const uint8_t *)a.logits + (long long)row * a.stride * (16 / E);
  // whole vectors from the first 16-byte border; the elements before and behind them
  // one by one
  const int head = min((int)(-(uintptr_t)x & 15u) / (16 / E), a.vocab), vecs = (a.vocab - head) / E;
  const int edges = a.vocab - vecs * E;
  const i32x4 *body = (const i32x4 *)(x + head * (16 / E));

  auto unpack = [&](const i32x4 &u, float *v) MOE_INLINE {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) {
        v[2 * j] = __uint_as_float((uint32_t)u[j] << 16);
        v[2 * j + 1] = __uint_as_float((uint32_t)u[j] & 0xFFFF0000u);
      } else {
        v[j] = __int_as_float(u[j]);
      }
    }
  };
  const int edge_at = tid < head ? tid : vecs * E + tid;   // of tid < edges
  auto edge = [&]() MOE_INLINE {
    return BF16 ? bf16_to_f32(((const uint16_t *)x)[edge_at]) : ((const float *)x)[edge_at];
  };

  // rounds of T vectors, U at once
  Sums sum = {kNegBig, 0.0f, 0.0f};
  int r = 0;
  for (; (r + U) * T <= vecs; r += U) {
    i32x4 u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) u[i] = body[(r + i) * T + tid];
    float v[U * E];
#pragma unroll
    for (int i = 0; i < U; ++i) unpack(u[i], v + i * E);
    add(sum, v);
  }
  if (r * T < vecs) {                            // the last: what is past the end is no logit
    i32x4 u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) u[i] = body[min((r + i) * T + tid, vecs - 1)];
    float v[U * E];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      unpack(u[i], v + i * E);
      if ((r + i) * T + tid >= vecs) {
#pragma unroll
        for (int j = 0; j < E; ++j) v[i * E + j] = -INFINITY;
      }
    }
    add(sum, v);
  }
  // (the threads' maxima leave the edges out, which all go into the list)
  const uint32_t own = sum.m > kNegBig ? order_of(sum.m) : 0u;
  if (tid < edges) {
    const float v[1] = {edge()};
    add(sum, v);
  }
  constexpr int GROUPS = LogprobLds<T, E>::groups;
  if (a.top) {
    uint32_t most = own;
#pragma unroll
    for (int m = 1; m < T / GROUPS; m <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, m, 64));
    if (tid % (T / GROUPS) == 0) s.most[tid / (T / GROUPS)] = most;
    if (tid == 0) s.owners = s.count = 0;
  }
  const Sums all = join_group<T / 64>(sum, s.red);         // (with the barrier behind the maxima)
  if (tid == T - 1) write_row(a, row, all);
  if (a.top == 0) return;

  // The n-th largest of the groups' maxima, by the first wave, bit by bit.
  if (tid < 64) {
    uint32_t m[GROUPS / 64], found = 0;
#pragma unroll
    for (int i = 0; i < GROUPS / 64; ++i) m[i] = s.most[64 * i + tid];
    for (int bit = 31; bit >= (BF16 ? 16 : 0); --bit) {
      const uint32_t trial = found | 1u << bit;
      int c = 0;
#pragma unroll
      for (int i = 0; i < GROUPS / 64; ++i) c += __popcll(__ballot(m[i] >= trial));
      if (c >= a.top) found = trial;
    }
    if (tid == 0) s.least = found;
  }
  __syncthreads();
  if (own >= s.least) s.owner[atomicAdd(&s.owners, 1)] = tid;
  uint64_t least = (uint64_t)s.least << 32;
  auto push = [&](float v, int i) MOE_INLINE {
    const uint64_t k = key_of(v, (uint32_t)i);
    if (k >= least) s.list[atomicAdd(&s.count, 1)] = k;
  };
  if (tid < edges) push(edge(), edge_at);
  __syncthreads();
  const int owners = s.owners, items = owners * ((vecs + T - 1) / T);
  auto vec_of = [&](int i) MOE_INLINE { return i < items ? i / owners * T + (int)s.owner[i % owners] : vecs; };
  int vec = vec_of(tid);
  i32x4 u = {};
  if (items > 0) u = body[min(vec, vecs - 1)];   // (a row of less than a vector has none)
  for (int i0 = 0; i0 < items; i0 += T) {
    // the next one is on its way while this one's go into the list
    const int next = vec_of(i0 + T + tid);
    const i32x4 un = body[min(next, vecs - 1)];
    if (vec < vecs) {
      float v[E];
      unpack(u, v);
#pragma unroll
      for (int j = 0; j < E; ++j) push(v[j], head + vec * E + j);
    }
    vec = next;
    u = un;
    __syncthreads();
    const int count = s.count;
    if (count > kList) least = prune(s, count, a.top);
    else __syncthreads();                        // all have read the count
  }
  // (the list holds at most kList keys, a.top at least: all of the row's that are not below `least`)
  const int count = s.count;
  for (int i = tid; i < count; i += T) {
    const uint64_t k = s.list[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += s.list[j] > k;
    if (rank < a.top) write_top(a, row, all, rank, k);
  }
}

// Threads of a row.  Rows too few to keep the CUs busy: up to 1024 (64 rows of 120832
// fp32: 15.2 us, 256 threads 21.2; 128 of 32003 bf16: 8.1 both; one of 8000 bf16: 64
// threads 7.2, 256 5.4, 1024 7.4).  Many: what the steps behind the pass cost counts
// (8192 rows of 1000 bf16: 64 threads 13.4 us, 256 31.7; of 8000: 34.6 and 35.5; 4096 of
// 120832 with 20 alternatives: 342 and 237, 1024 threads 236, with one 206, 196 and 227).
int threads_of_row(int rows, int vecs) {
  if (rows < 512) return vecs >= 8192 ? 1024 : vecs >= 512 ? 256 : 64;
  return vecs >= 1024 ? 256 : 64;
}

template <bool BF16>
hipError_t launch(const LogprobArgs &a, hipStream_t s) {
  const int vecs = a.vocab / (BF16 ? 8 : 4), threads = threads_of_row(a.rows, vecs);
  const long long most = max_groups(1024);
  for (long long row0 = 0; row0 < a.rows; row0 += most) {
    const unsigned rows = (unsigned)(a.rows - row0 < most ? a.rows - row0 : most);
    if (threads == 1024) logprob_kernel<BF16, 1024><<<rows, 1024, 0, s>>>(a, (int)row0);
    else if (threads == 256) logprob_kernel<BF16, 256><<<rows, 256, 0, s>>>(a, (int)row0);
    else logprob_kernel<BF16, 64><<<rows, 64, 0, s>>>(a, (int)row0);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_logprobs(const LogprobArgs &a, hipStream_t s) {
  return a.is_bf16 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
