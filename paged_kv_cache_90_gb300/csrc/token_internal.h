// token_internal.h — launch parameters and launchers of the calls around a step's new
// tokens (rotary and quantising cache writes, read back, attention of drafted trees and
// over token-scaled caches).  Not part of the public ABI.
#pragma once

#include "pkv_internal.h"

namespace pkv {

constexpr int kI8 = 5;  // PKV_I8, beside DType's codes

// ---- rotary_and_cache, quantize_and_cache, read_cache ----------------------------------
struct TokenParams {
  CacheWriteParams w;          // key / value, caches, slots (no amax)
  float* k_token_scales;       // i8 cache: [NB, Hk, bs] scales (or null)
  float* v_token_scales;
  int64_t ts_block, ts_head;   // their strides, elements
  const void* query;           // [T, Hq, D], the key's dtype
  void* query_out;
  int64_t q_stride_t, q_stride_h, qo_stride_t, qo_stride_h;
  int num_heads;               // 0: no query
  const void* positions;       // [T]
  bool positions64;
  int rotary_dim;              // 0: no rotation
  bool interleaved;
  float magnitude;
  // pair i turns by turns[i] / 2^64 + turns_low[i] / 2^96 of a circle per position
  uint64_t turns[64];
  uint32_t turns_low[64];
};
cudaError_t launch_token_write(const TokenParams& p, cudaStream_t stream);
cudaError_t launch_token_read(const TokenParams& p, cudaStream_t stream);

// ---- attention of drafted trees / decode over token-scaled caches -----------------------
struct TreeParams {
  void* out;                   // [T, Hq, D]
  const void* query;
  int q_dtype;                 // and out's
  int64_t out_stride_t, out_stride_h, q_stride_t, q_stride_h;
  const void* key_cache;       // [NB, Hk, bs, D]
  const void* value_cache;
  int kv_dtype;
  int64_t cs_block, cs_head;   // elements
  const float* k_token_scales; // i8 cache: [NB, Hk, bs]
  const float* v_token_scales;
  int64_t ts_block, ts_head;
  const float* k_head_scales;  // e4m3 cache: [Hk] (or null)
  const float* v_head_scales;
  const int32_t* block_tables;
  int64_t bt_stride;
  const int32_t* context_lens;
  const int32_t* query_start_loc;  // null: one row per sequence
  const int64_t* tree_mask;        // null: rows see the whole context (with the window)
  int64_t mask_stride;
  int mask_words;
  int num_seqs, num_tokens, num_heads, num_kv_heads, group, head_dim, block_size, max_blocks_per_seq;
  int64_t num_blocks;
  float qk_scale_log2;         // scale * log2(e) * k_scale
  float v_scale;
  int sliding_window;
  unsigned int* err;
};
cudaError_t launch_tree_core(const TreeParams& p, cudaStream_t stream);  // CUDA cores, any call

// The tensor-core kernel's split of the work over `grid` blocks.
struct TreeSplit {
  // the item that begins in a block's range and goes on behind it: its nodes (0: there is
  // none), first query row, KV head and the last block that holds a part of it
  struct Tail {
    int nodes, row0, kvh, last;
  };
  static constexpr size_t kMaxSms = 240;
  static constexpr size_t kMaxGrid = 3 * kMaxSms;                     // blocks
  static constexpr size_t kHeader = kWorkspaceHeader + kMaxGrid * sizeof(Tail);  // (a multiple of 256)
  int grid;
  int rows;     // rows of a part's slot
  int tq;       // nodes of a row tile: 128 / group
  int item_nodes;  // nodes of an item
  int q_nodes;  // nodes of one query copy
  int bs_shift; // log2 of the block size
  bool out_vec;      // output rows are 8-byte aligned
  bool vec_scales;   // four tokens' scales are 16 aligned bytes
  Tail* tails;  // [grid]
  float* o;     // [2 grid, rows, D]: block b's part of an item begun before it, then of its own
  float2* ml;   // [2 grid, rows] maximum (base 2) and sum
};
bool tree_tc_supported(const TreeParams& p);  // bf16 caches (tree_tc.cu)
bool tree_i8_supported(const TreeParams& p);  // token-scaled caches (tree_i8.cu)
bool tree_tensor_supported(const TreeParams& p);
bool decode_i8_supported(const TreeParams& p);  // one row a sequence, few heads (decode_i8.cu)
int decode_i8_blocks_per_sm(int group);
int tree_part_rows(int64_t num_tokens, int group, bool decode, bool one_tile);
size_t tree_workspace(int grid, int rows, int head_dim);
cudaError_t launch_tree_tensor(const TreeParams& p, int grid, int rows, void* ws, cudaStream_t stream);
cudaError_t launch_tree_i8(const TreeParams& p, TreeSplit sp, cudaStream_t stream);
cudaError_t launch_decode_i8(const TreeParams& p, TreeSplit sp, cudaStream_t stream);
cudaError_t launch_tree_merge(const TreeParams& p, const TreeSplit& sp, cudaStream_t stream);

}  // namespace pkv
