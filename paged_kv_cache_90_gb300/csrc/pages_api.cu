// pages_api.cu — the C ABI's calls over the caches of all layers (declared in include/pkv.h):
// blocks copied, accepted drafted tokens moved.  Argument checks and launch parameters only.
#include <algorithm>

#include "pages_internal.h"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kMaxCaches = 1024;

// Checks the list; all its caches share num_blocks and block_size.
pkv_status check_list(const pkv_tensor* const* caches, int32_t n) {
  if (!caches) return fail(PKV_ERR_INVALID_ARG, "caches: null pointer");
  if (n < 1 || n > kMaxCaches) return fail(PKV_ERR_INVALID_ARG, "num_caches must be 1 to %d", kMaxCaches);
  for (int i = 0; i < n; ++i) {
    const pkv_status st = check_pages(caches[i], "cache");
    if (st) return st;
    if (caches[i]->shape[0] != caches[0]->shape[0] || caches[i]->shape[2] != caches[0]->shape[2])
      return fail(PKV_ERR_INVALID_ARG, "cache %d: all caches must have the same num_blocks and block_size", i);
    if (caches[i]->shape[1] > 65535) return fail(PKV_ERR_UNSUPPORTED, "too many heads");
  }
  return PKV_OK;
}

// Caches first .. of the list, as many as a launch takes, those without a KV head left out;
// returns where the next launch starts.
int fill(const pkv_tensor* const* caches, int n, int first, PagesParams* pp) {
  PagesParams& p = *pp;
  p.num_caches = 0;
  p.first_chunk[0] = 0;
  p.num_blocks = caches[0]->shape[0];
  int i = first;
  for (; i < n && p.num_caches < kPageCaches; ++i) {
    const pkv_tensor* t = caches[i];
    if (t->shape[1] == 0) continue;
    const int eb = elt_bytes(t->dtype);
    PageCache& c = p.caches[p.num_caches];
    c.base = static_cast<unsigned char*>(t->data);
    c.block_stride = t->stride[0] * eb;
    c.head_stride = t->stride[1] * eb;
    c.heads = uint32_t(t->shape[1]);
    c.row_bytes = uint32_t((t->ndim == 3 ? 1 : t->shape[3]) * eb);
    const int64_t tile = t->shape[2] * c.row_bytes;
    const bool joined = c.heads == 1 || c.head_stride == tile;  // a block's heads lie together
    c.run_bytes = uint32_t(joined ? c.heads * tile : tile);     // (at most 65535 heads of 16 KB)
    c.run_stride = joined ? 0 : c.head_stride;
    c.vec = 16;
    const int64_t chunks = (int64_t(c.run_bytes) + kPageChunk - 1) / kPageChunk * (joined ? 1 : c.heads);
    p.first_chunk[p.num_caches + 1] = p.first_chunk[p.num_caches] + uint32_t(chunks);
    ++p.num_caches;
  }
  return i;
}

// 16 bytes at a time where every address is a multiple of them (`row`: of each token's row too).
void choose_vectors(PagesParams* p, bool row) {
  for (int i = 0; i < p->num_caches; ++i) {
    PageCache& c = p->caches[i];
    const int64_t all = int64_t(reinterpret_cast<uintptr_t>(c.base)) | c.block_stride | c.head_stride |
                        (row ? c.row_bytes : c.run_bytes);
    c.vec = all % 16 == 0 ? 16 : 4;
  }
}

pkv_status check_i32(const pkv_tensor* t, const char* name, int64_t n) {
  pkv_status st;
  if ((st = check_basic(t, name, 1)) || (st = check_dtype(t, name, PKV_I32))) return st;
  if (n >= 0 && t->shape[0] != n) return fail(PKV_ERR_INVALID_ARG, "%s must hold %lld numbers", name, (long long)n);
  if (t->shape[0] > 1 && t->stride[0] != 1) return fail(PKV_ERR_INVALID_ARG, "%s must be contiguous", name);
  if (reinterpret_cast<uintptr_t>(t->data) & 3) return fail(PKV_ERR_INVALID_ARG, "%s must be 4-byte aligned", name);
  return PKV_OK;
}

// Whether int32 arrays share memory (`a` contiguous; `b` may be a table).
bool overlap(const pkv_tensor* a, const pkv_tensor* b) {
  if (a->shape[0] == 0 || b->shape[0] == 0) return false;
  const int64_t n = (b->shape[0] - 1) * b->stride[0] + (b->ndim == 2 ? b->shape[1] : 1);
  const uintptr_t x = reinterpret_cast<uintptr_t>(a->data), y = reinterpret_cast<uintptr_t>(b->data);
  return x < y + 4 * n && y < x + 4 * a->shape[0];
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_copy_cache_blocks(const pkv_tensor* const* caches, int32_t num_caches, const pkv_tensor* src_dst_pairs,
                                 pkv_stream stream) {
  pkv_status st;
  if ((st = check_list(caches, num_caches)) || (st = check_pairs(src_dst_pairs))) return st;
  const int64_t n = src_dst_pairs->shape[0];
  if (n > 0x7fffffff) return fail(PKV_ERR_UNSUPPORTED, "too many pairs");
  if (dry_run() || n == 0) return PKV_OK;
  DeviceState* s;
  if ((st = device_state(&s))) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int64_t* pairs = static_cast<const int64_t*>(src_dst_pairs->data);
  PagesParams p;
  p.err = s->err;
  cudaError_t e = cudaSuccess;
  if (debug_sync()) {  // O(pairs^2) device check, debug only
    CopyBlocksParams check{};
    check.pairs = pairs;
    check.num_pairs = n;
    check.err = s->err;
    e = launch_copy_pairs_check(check, cs);
  }
  for (int first = 0; first < num_caches && e == cudaSuccess;) {
    first = fill(caches, num_caches, first, &p);
    choose_vectors(&p, false);
    if (p.num_caches) e = launch_copy_pages(p, pairs, n, cs);
  }
  return finish_call(s, e, cs, "copy_cache_blocks");
}

pkv_status pkv_keep_tokens(const pkv_tensor* const* caches, int32_t num_caches, const pkv_tensor* block_tables,
                           const pkv_tensor* context_lens, const pkv_tensor* query_start_loc, const pkv_tensor* keep,
                           const pkv_tensor* keep_counts, const pkv_tensor* new_lens, int32_t block_size,
                           int32_t max_blocks_per_seq, pkv_stream stream) {
  pkv_status st;
  if ((st = check_list(caches, num_caches)) || (st = check_basic(block_tables, "block_tables", 2)) ||
      (st = check_dtype(block_tables, "block_tables", PKV_I32)))
    return st;
  const int64_t S = block_tables->shape[0];
  if (reinterpret_cast<uintptr_t>(block_tables->data) & 3)
    return fail(PKV_ERR_INVALID_ARG, "block_tables must be 4-byte aligned");
  if ((st = check_i32(context_lens, "context_lens", S)) || (st = check_i32(query_start_loc, "query_start_loc", S + 1)) ||
      (st = check_i32(keep, "keep", -1)) || (st = check_i32(keep_counts, "keep_counts", S)) ||
      (new_lens && (st = check_i32(new_lens, "new_lens", S))))
    return st;
  if (caches[0]->shape[2] != block_size) return fail(PKV_ERR_INVALID_ARG, "block_size must match the caches");
  if (block_tables->shape[1] != max_blocks_per_seq || max_blocks_per_seq < 1)
    return fail(PKV_ERR_INVALID_ARG, "block_tables must be [num_seqs, max_blocks_per_seq]");
  if (new_lens)
    for (const pkv_tensor* in : {context_lens, query_start_loc, keep, keep_counts, block_tables})
      if (overlap(new_lens, in))
        return fail(PKV_ERR_INVALID_ARG, "new_lens must share no memory with an input (all blocks of the launch read them)");
  if (int64_t(max_blocks_per_seq) * block_size > (int64_t(1) << 30))
    return fail(PKV_ERR_UNSUPPORTED, "max context above 2^30 tokens");
  if (S > 65535 || keep->shape[0] > (1 << 28))
    return fail(PKV_ERR_UNSUPPORTED, "num_seqs must be <= 65535, num_tokens <= 2^28");
  // a cache that is listed twice would be moved twice, by blocks that run at the same time
  const void* seen[kMaxCaches];
  for (int i = 0; i < num_caches; ++i) seen[i] = caches[i]->data;
  std::sort(seen, seen + num_caches);
  for (int i = 1; i < num_caches; ++i)
    if (seen[i] && seen[i] == seen[i - 1]) return fail(PKV_ERR_INVALID_ARG, "a cache is listed twice");
  if (dry_run() || S == 0) return PKV_OK;
  DeviceState* s;
  if ((st = device_state(&s))) return st;
  KeepParams k{};
  k.block_tables = static_cast<const int32_t*>(block_tables->data);
  k.bt_stride = block_tables->stride[0];
  k.context_lens = static_cast<const int32_t*>(context_lens->data);
  k.query_start_loc = static_cast<const int32_t*>(query_start_loc->data);
  k.keep = static_cast<const int32_t*>(keep->data);
  k.keep_counts = static_cast<const int32_t*>(keep_counts->data);
  k.new_lens = new_lens ? static_cast<int32_t*>(new_lens->data) : nullptr;
  k.num_seqs = int(S);
  k.num_tokens = int(keep->shape[0]);
  k.block_size = block_size;
  k.max_blocks_per_seq = max_blocks_per_seq;
  k.err = s->err;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  PagesParams p;
  p.err = s->err;
  cudaError_t e = cudaSuccess;
  k.report = true;
  for (int first = 0; first < num_caches && e == cudaSuccess;) {
    first = fill(caches, num_caches, first, &p);
    choose_vectors(&p, true);
    if (!p.num_caches && !k.report) continue;  // (caches without heads: new_lens is written all the same)
    e = launch_keep_tokens(p, k, cs);
    k.report = false;
  }
  return finish_call(s, e, cs, "keep_tokens");
}

}  // extern "C"
