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
// that there are no ties, and the list's own order does not matter.
//
// Bound by memory.  Few rows are cut into parts, which a second launch joins.
#include "block_common.hpp"

namespace moe {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
constexpr int kTop = kLogprobTop;
constexpr int kList = 512;                       // keys that are ranked by counting
constexpr int kSweep = 2048;                     // keys that one sweep adds at most
static_assert(kTop <= 64 && kLogprobParts * kTop <= kSweep, "keys of a list");

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
__device__ __forceinline__ Sums join(const Sums &a, const Sums &b) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  const float da = apart(a.m, r.m), db = apart(b.m, r.m);
  const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
  r.l = a.l * fa + b.l * fb;
  r.t = fmaf(a.l, da, a.t) * fa + fmaf(b.l, db, b.t) * fb;
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
// The sums of all 256 threads, in every thread.
__device__ __forceinline__ Sums join_group(Sums s, Sums *red) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1)
    s = join(s, Sums{__shfl_xor(s.m, m, 64), __shfl_xor(s.l, m, 64), __shfl_xor(s.t, m, 64)});
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  return join(join(red[0], red[1]), join(red[2], red[3]));
}

struct __align__(16) LogprobLds {
  uint64_t list[kList + kSweep];
  uint32_t most[256];            // order of each thread's maximum
  Sums red[4];
  uint32_t owner[256];
  int owners, count, tally[2];
  uint32_t least;
};

// The n-th largest of the list's `count` keys (n <= count; keys differ): bit by bit.
__device__ __forceinline__ uint64_t nth_largest(LogprobLds &s, int count, int n) {
  constexpr int PER = (kList + kSweep) / 256;
  uint64_t k[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) k[i] = i * 256 + (int)threadIdx.x < count ? s.list[i * 256 + threadIdx.x] : 0;
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
__device__ __forceinline__ uint64_t prune(LogprobLds &s, int count, int n) {
  constexpr int PER = (kList + kSweep) / 256;
  const uint64_t least = nth_largest(s, count, n);
  uint64_t k[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) k[i] = i * 256 + (int)threadIdx.x < count ? s.list[i * 256 + threadIdx.x] : 0;
  __syncthreads();
  if (threadIdx.x == 0) s.count = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (k[i] >= least) s.list[atomicAdd(&s.count, 1)] = k[i];
  __syncthreads();
  return least;
}
// put(place, key) for the n largest keys of the list (fewer if it holds fewer), which
// is complete behind a barrier.
template <typename Put>
__device__ __forceinline__ void ranked(LogprobLds &s, int n, Put &&put) {
  if (s.count > kList) prune(s, s.count, n);
  const int count = s.count;
  for (int i = threadIdx.x; i < count; i += 256) {
    const uint64_t k = s.list[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += s.list[j] > k;
    if (rank < n) put(rank, k);
  }
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

// Part blockIdx % parts of row first + blockIdx / parts.
template <bool BF16>
__global__ __launch_bounds__(256) void logprob_kernel(LogprobArgs a, int first) {
  __shared__ LogprobLds s;
  constexpr int E = BF16 ? 8 : 4, U = 4;         // elements of a vector, vectors at once
  const int tid = threadIdx.x, part = (int)(blockIdx.x % (uint32_t)a.parts);
  const int row = first + (int)(blockIdx.x / (uint32_t)a.parts);
  const uint8_t *x = (const uint8_t *)a.logits + (long long)row * a.stride * (16 / E);
  // whole vectors from the first 16-byte border; the elements before and behind them
  // (part 0) one by one
  const int head = min((int)(-(uintptr_t)x & 15u) / (16 / E), a.vocab), vecs = (a.vocab - head) / E;
  const int edges = part == 0 ? a.vocab - vecs * E : 0;
  const i32x4 *body = (const i32x4 *)(x + head * (16 / E));
  // this part's rounds of 256 vectors
  const int rounds = (vecs + 255) / 256;
  const int r0 = (int)((long long)rounds * part / a.parts), r1 = (int)((long long)rounds * (part + 1) / a.parts);

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
  auto edge_at = [&]() MOE_INLINE { return tid < head ? tid : vecs * E + tid; };     // of tid < edges
  auto edge = [&](int i) MOE_INLINE {
    return BF16 ? bf16_to_f32(((const uint16_t *)x)[i]) : ((const float *)x)[i];
  };

  Sums sum = {kNegBig, 0.0f, 0.0f};
  int r = r0;
  for (; (r + U - 1) * 256 + 255 < vecs && r + U <= r1; r += U) {
    i32x4 u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) u[i] = body[(r + i) * 256 + tid];
    float v[U * E];
#pragma unroll
    for (int i = 0; i < U; ++i) unpack(u[i], v + i * E);
    add(sum, v);
  }
  for (; r < r1; ++r)
    if (r * 256 + tid < vecs) {
      float v[E];
      unpack(body[r * 256 + tid], v);
      add(sum, v);
    }
  // (the threads' maxima leave the edges out, which all go into the list)
  const uint32_t own = sum.m > kNegBig ? order_of(sum.m) : 0u;
  if (tid < edges) {
    const float v[1] = {edge(edge_at())};
    add(sum, v);
  }
  const Sums all = join_group(sum, s.red);

  uint64_t *keys = nullptr;
  if (a.parts > 1) {
    const long long unit = (long long)row * a.parts + part;
    if (tid == 0) *(float4 *)(a.ws + unit * 16) = make_float4(all.m, all.l, all.t, 0.0f);
    keys = (uint64_t *)(a.ws + (long long)a.rows * a.parts * 16) + unit * a.top;
  } else if (tid == 0) {
    write_row(a, row, all);
  }
  if (a.top == 0) return;

  // The n-th largest of the threads' maxima, by the first wave, bit by bit.
  s.most[tid] = own;
  if (tid == 0) s.owners = s.count = 0;
  __syncthreads();
  if (tid < 64) {
    const uint4 m = *(const uint4 *)&s.most[4 * tid];
    uint32_t found = 0;
    for (int bit = 31; bit >= (BF16 ? 16 : 0); --bit) {
      const uint32_t trial = found | 1u << bit;
      const int c = __popcll(__ballot(m.x >= trial)) + __popcll(__ballot(m.y >= trial)) +
                    __popcll(__ballot(m.z >= trial)) + __popcll(__ballot(m.w >= trial));
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
  if (tid < edges) push(edge(edge_at()), edge_at());
  __syncthreads();
  const int owners = s.owners, items = owners * (r1 - r0);
  for (int i0 = 0; i0 < items; i0 += 256) {
    const int i = i0 + tid, vec = i < items ? (r0 + i / owners) * 256 + (int)s.owner[i % owners] : vecs;
    if (vec < vecs) {
      float v[E];
      unpack(body[vec], v);
#pragma unroll
      for (int j = 0; j < E; ++j) push(v[j], head + vec * E + j);
    }
    __syncthreads();
    const int count = s.count;
    if (count > kList) least = prune(s, count, a.top);
    else __syncthreads();                        // all have read the count
  }
  if (a.parts == 1) {
    ranked(s, a.top, [&](int place, uint64_t key) { write_top(a, row, all, place, key); });
  } else {
    const int count = s.count;
    if (tid < a.top && tid >= count) keys[tid] = 0;
    ranked(s, a.top, [&](int place, uint64_t key) { keys[place] = key; });
  }
}

// The parts of a row together.
__global__ __launch_bounds__(256) void logprob_join_kernel(LogprobArgs a) {
  __shared__ LogprobLds s;
  const int tid = threadIdx.x, row = blockIdx.x;
  Sums all = {kNegBig, 0.0f, 0.0f};
  if (tid < a.parts) {
    const float4 f = *(const float4 *)(a.ws + ((long long)row * a.parts + tid) * 16);
    all = {f.x, f.y, f.z};
  }
  if (tid == 0) s.count = 0;
  all = join_group(all, s.red);
  if (tid == 0) write_row(a, row, all);
  const uint64_t *keys = (const uint64_t *)(a.ws + (long long)a.rows * a.parts * 16) + (long long)row * a.parts * a.top;
  for (int i = tid; i < a.parts * a.top; i += 256) {
    const uint64_t k = keys[i];
    if (k) s.list[atomicAdd(&s.count, 1)] = k;
  }
  __syncthreads();
  if (a.top) ranked(s, a.top, [&](int place, uint64_t key) { write_top(a, row, all, place, key); });
}

// Parts of a row: about 1024 workgroups, of 4 rounds of vectors each at least.
int logprob_parts(int rows, int vocab, int is_bf16) {
  const int rounds = vocab / (256 * (is_bf16 ? 8 : 4));
  int p = 1024 / (rows > 0 ? rows : 1);
  p = p < rounds / 4 ? p : rounds / 4;
  return p < 1 ? 1 : p > kLogprobParts ? kLogprobParts : p;
}

hipError_t launch_logprobs(const LogprobArgs &a, hipStream_t s) {
  const long long most = max_groups(256) / a.parts;
  for (long long row0 = 0; row0 < a.rows; row0 += most) {
    const long long rows = a.rows - row0 < most ? a.rows - row0 : most;
    const unsigned grid = (unsigned)(rows * a.parts);
    if (a.is_bf16) logprob_kernel<true><<<grid, 256, 0, s>>>(a, (int)row0);
    else logprob_kernel<false><<<grid, 256, 0, s>>>(a, (int)row0);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (a.parts > 1) logprob_join_kernel<<<(unsigned)a.rows, 256, 0, s>>>(a);     // (of 1024 rows at most)
  return hipGetLastError();
}

}  // namespace moe
