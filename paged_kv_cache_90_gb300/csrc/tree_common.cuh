// tree_common.cuh — what the attention kernels for drafted trees (and for decode over a
// token-scaled cache) share: a sequence's checked extent and its masks.
#pragma once

#include "device_common.cuh"
#include "token_internal.h"

namespace pkv {
namespace tree {

// A sequence's work: n query rows from row q0 of the batch on, over positions lo .. L - 1,
// of which those from P = L - n on are drafted nodes hidden by masks (with no mask, P = L).
struct Extent {
  int q0, n, L, P, lo;
};

// Sequence s's extent; n = 0 if it has no rows or is out of range (*bad tells which).
__device__ __forceinline__ Extent extent(const TreeParams& p, int s, bool* bad) {
  Extent e;
  e.L = __ldg(p.context_lens + s);
  e.lo = 0;
  if (p.query_start_loc) {
    e.q0 = __ldg(p.query_start_loc + s);
    e.n = __ldg(p.query_start_loc + s + 1) - e.q0;
  } else {
    e.q0 = s;
    e.n = 1;
  }
  const int max_ctx = p.max_blocks_per_seq * p.block_size;
  *bad = e.n != 0 && (e.L < 0 || e.L > max_ctx || e.n < 0 || e.q0 < 0 || e.q0 > p.num_tokens - e.n ||
                      (p.tree_mask && (e.n > e.L || e.n > 64 * p.mask_words)));
  if (*bad) e.n = 0;
  e.P = e.L;
  if (e.n && p.tree_mask)
    e.P = e.L - e.n;
  else if (e.n)
    e.lo = window_start(e.L, p.sliding_window);
  return e;
}

// Whether the row whose masks start at `mask` attends to drafted node c (0 <= c < n).
__device__ __forceinline__ bool sees_node(const int64_t* mask, int c) {
  return (uint64_t(__ldg(mask + (c >> 6))) >> (c & 63)) & 1;
}

}  // namespace tree
}  // namespace pkv
