// pages_internal.h — launch parameters and launchers of the calls over many caches
// (pages.cu).  Not part of the public ABI.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// A cache, or a scale array, as bytes.
struct PageCache {
  unsigned char* base;
  int64_t block_stride, head_stride;  // bytes
  int64_t run_stride;                 // between a block's contiguous runs
  uint32_t run_bytes;                 // of a run: all heads of a block where they lie together, or one
  uint32_t row_bytes;                 // of a (token, KV head)
  uint32_t heads;
  uint32_t vec;                       // bytes of an access: 16 or 4
};

constexpr int kPageCaches = 96;       // of a launch: they travel in its parameters
constexpr int kPageChunk = 16384;     // bytes that a thread block copies

struct PagesParams {
  PageCache caches[kPageCaches];
  uint32_t first_chunk[kPageCaches + 1];  // (copies) chunks of a block in the caches before this one
  int num_caches;
  int64_t num_blocks;
  unsigned int* err;
};
cudaError_t launch_copy_pages(const PagesParams& p, const int64_t* pairs, int64_t num_pairs, cudaStream_t stream);

struct KeepParams {
  const int32_t* block_tables;
  int64_t bt_stride;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  const int32_t* keep;
  const int32_t* keep_counts;
  int32_t* new_lens;  // or null
  bool report;        // the launch that writes new_lens and reports errors (of a call's several)
  int num_seqs, num_tokens, block_size, max_blocks_per_seq;
  unsigned int* err;
};
cudaError_t launch_keep_tokens(const PagesParams& p, const KeepParams& k, cudaStream_t stream);

}  // namespace pkv
