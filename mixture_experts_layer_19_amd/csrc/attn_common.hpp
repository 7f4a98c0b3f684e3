// attn_common.hpp -- what the attention kernels share: which keys a query row
// sees, the order in which key tiles are visited, loads of keys and queries.
//
//   out[r, h] = sum_j softmax_j(scale * q[r, h] . k[j, h / group]) v[j, h / group]
//
// over the keys j <= pos(r) of the row's sequence; with a window W also
// j > pos(r) - W or j < sinks.  A row that sees no key gives zeros.  Scores,
// maxima, sums and the output accumulate in fp32; the softmax runs on powers
// of two (scale * log2(e) is folded into the scores).
//
// The rows of one sequence and KV head are the pairs (token, query head of
// the group), token-major: row m is token m / group, head m % group.  So the
// query heads that share keys fill a matrix tile together.
#pragma once
#include "block_common.hpp"

namespace moe {

// Key tiles of BK keys that tokens [i0, i1] of a sequence visit: the tiles
// that hold sinks, then those of the window.
template <int BK>
struct KeyRange {
  int sink_tiles, first, tiles;
  __device__ __forceinline__ KeyRange(const SeqGeo &g, int i0, int i1, int window, int sinks) {
    const int hi = min(max(g.pos0 + i1 + 1, 0), g.len);
    const int lo = window ? min(max(g.pos0 + i0 - window + 1, 0), hi) : 0;
    first = lo / BK;
    sink_tiles = window ? min((min(sinks, hi) + BK - 1) / BK, first) : 0;
    tiles = sink_tiles + (hi + BK - 1) / BK - first;
  }
  __device__ __forceinline__ int key(int t) const {   // first key of the t-th tile
    return (t < sink_tiles ? t : first + t - sink_tiles) * BK;
  }
};

// Keys that one query row sees: [lo, hi) and [0, sinks).
struct RowMask {
  int lo, hi, sinks;
  __device__ __forceinline__ RowMask(const SeqGeo &g, int token, bool in, int window, int nsinks) {
    const int pos = g.pos0 + token;
    hi = in ? min(pos + 1, g.len) : 0;
    lo = window ? pos - window + 1 : 0;
    sinks = nsinks;
  }
  __device__ __forceinline__ bool sees(int key) const { return key < hi && (key >= lo || key < sinks); }
};

}  // namespace moe
