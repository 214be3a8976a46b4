// pages.cu — pages of many caches at once: blocks copied in the caches of all layers
// (copy_cache_blocks) and the drafted tokens that were accepted moved together (keep_tokens).
//
// Both move bytes and nothing else: HBM bounds the large calls (twice the moved bytes) and the
// launch the small ones, which is why one launch takes the caches of all layers: their descriptors
// travel in its parameters.  150 blocks of 16 tokens, 8 heads of 128 in bf16, in 32 caches (157 MB read, as
// much written): 49 us, 6.4 TB/s, with one pool or several in turn.  Three blocks in 8 caches: 1.9 us of the GPU's time, 5.7 of the
// caller's.  48 sequences that keep some of their 8 to 24 drafted tokens in 24 int8 caches and their
// scales: 5.8 us of the GPU's time (four round trips: lengths, kept nodes, table entries, rows), 10
// of the caller's.
#include "device_common.cuh"
#include "pages_internal.h"

namespace pkv {

namespace {

constexpr int kCopyThreads = 256, kInFlight = 4;  // 16-byte loads that a thread has in flight

__device__ __forceinline__ uint4 load_once(const unsigned char* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

// A thread block copies one chunk of at most kPageChunk bytes of a (pair, cache): consecutive
// blocks take consecutive chunks, then the next cache, then the next pair.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ PagesParams p,
                                                                  const int64_t* pairs, int64_t first_pair) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const uint32_t chunks = p.first_chunk[p.num_caches];
  const uint32_t at = blockIdx.x % chunks;
  const int64_t pair = first_pair + blockIdx.x / chunks;
  const int64_t src = pairs[2 * pair], dst = pairs[2 * pair + 1];
  if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
    if (threadIdx.x == 0 && at == 0) raise_device_error(p.err, kErrCopyPair);
    return;
  }
  int a = 0, b = p.num_caches;  // the cache: first_chunk[a] <= at < first_chunk[b]
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (p.first_chunk[m] <= at) a = m; else b = m;
  }
  const PageCache c = p.caches[a];
  // the chunk's run (a whole block of the cache, or one head of it) and its place in the run
  const uint32_t per_run = (c.run_bytes + kPageChunk - 1) / kPageChunk;
  const uint32_t i = at - p.first_chunk[a], run = i / per_run, from = (i - run * per_run) * kPageChunk;
  const uint32_t bytes = min(uint32_t(kPageChunk), c.run_bytes - from);
  const unsigned char* s = c.base + src * c.block_stride + int64_t(run) * c.run_stride + from;
  unsigned char* d = c.base + dst * c.block_stride + int64_t(run) * c.run_stride + from;
  if (c.vec == 16) {
    const uint32_t step = kCopyThreads * 16;
    for (uint32_t o = threadIdx.x * 16; o < bytes; o += kInFlight * step) {
      uint4 v[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u)
        if (o + u * step < bytes) v[u] = load_once(s + o + u * step);
#pragma unroll
      for (int u = 0; u < kInFlight; ++u)
        if (o + u * step < bytes) *reinterpret_cast<uint4*>(d + o + u * step) = v[u];
    }
  } else {
    for (uint32_t o = threadIdx.x * 4; o < bytes; o += kCopyThreads * 4)
      *reinterpret_cast<uint32_t*>(d + o) = *reinterpret_cast<const uint32_t*>(s + o);
  }
}

constexpr int kKeepThreads = 128;
constexpr int kKeepBatch = 64;  // kept tokens whose places are in shared memory at a time
constexpr int kKeepLoads = 4;   // of a thread in flight

// Block (s, c): sequence s in cache c.  A thread has columns (a vector of one KV head's row) of its
// own and takes the kept tokens in ascending order, kKeepLoads loads and then their stores.  Token i
// goes from place a_i to place i <= a_i, so a load never follows the store that overwrites it: that
// is token a_i's own, and a_i = j > i comes later.
__global__ void __launch_bounds__(kKeepThreads) keep_tokens_kernel(const __grid_constant__ PagesParams p,
                                                                   const __grid_constant__ KeepParams k) {
  __shared__ int64_t from[kKeepBatch], to[kKeepBatch];  // block << 8 | place in it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int s = blockIdx.x, tid = threadIdx.x;
  const int q0 = k.query_start_loc[s], q1 = k.query_start_loc[s + 1], L = k.context_lens[s], kept = k.keep_counts[s];
  const int n = int(uint32_t(q1) - uint32_t(q0)), P = int(uint32_t(L) - uint32_t(n));
  const bool first_cache = blockIdx.y == 0 && k.report;
  const int64_t room = int64_t(k.max_blocks_per_seq) * k.block_size;
  // (n and P may wrap where the numbers are nonsense; they are used behind this check)
  if (q0 < 0 || q1 < q0 || q1 > k.num_tokens || L < 0 || L > room || n > L) {
    if (tid == 0 && first_cache) raise_device_error(k.err, kErrContextLen);
    return;
  }
  bool bad = kept < 0 || kept > n, bad_entry = false;
  const int32_t* keep = k.keep + q0;
  const int32_t* table = k.block_tables + int64_t(s) * k.bt_stride;
  const int shift = 31 - __clz(k.block_size), mask = k.block_size - 1;
  auto place = [&](int node) -> int64_t {
    const int pos = P + node;
    const int32_t blk = table[pos >> shift];
    if (blk < 0 || int64_t(blk) >= p.num_blocks) bad_entry = true;
    return int64_t(blk) << 8 | (pos & mask);
  };
  if (!bad)
    for (int i = tid; i < kept; i += kKeepThreads) {
      const int a = keep[i], before = i ? keep[i - 1] : -1;
      if (a <= before || a >= n || a < i) {
        bad = true;
      } else if (a != i) {
        (void)place(a);
        (void)place(i);
      }
    }
  const bool any_bad = __syncthreads_or(bad), any_entry = __syncthreads_or(bad_entry);
  if (any_bad || any_entry) {
    if (tid == 0 && first_cache) raise_device_error(k.err, any_bad ? kErrKeep : kErrTableEntry);
    return;
  }
  if (first_cache && tid == 0 && k.new_lens) k.new_lens[s] = P + kept;
  if (int(blockIdx.y) >= p.num_caches) return;
  const PageCache c = p.caches[blockIdx.y];
  const int per_head = c.row_bytes / c.vec, columns = c.heads * per_head;
  for (int i0 = 0; i0 < kept; i0 += kKeepBatch) {
    const int m = min(kKeepBatch, kept - i0);
    __syncthreads();  // (the batch before has been read)
    if (tid < m) {
      const int a = keep[i0 + tid];
      from[tid] = a == i0 + tid ? -1 : place(a);  // (it stays)
      to[tid] = a == i0 + tid ? -1 : place(i0 + tid);
    }
    __syncthreads();
    for (int col = tid; col < columns; col += kKeepThreads) {
      const int h = col / per_head;
      unsigned char* base = c.base + int64_t(h) * c.head_stride + (col - h * per_head) * c.vec;
      auto at = [&](int64_t x) { return base + (x >> 8) * c.block_stride + int64_t(x & 255) * c.row_bytes; };
      for (int i = 0; i < m; i += kKeepLoads) {
        uint4 v[kKeepLoads];
#pragma unroll
        for (int u = 0; u < kKeepLoads; ++u) {
          if (i + u >= m || from[i + u] < 0) continue;
          const unsigned char* x = at(from[i + u]);
          if (c.vec == 16) v[u] = *reinterpret_cast<const uint4*>(x);
          else v[u].x = *reinterpret_cast<const uint32_t*>(x);
        }
#pragma unroll
        for (int u = 0; u < kKeepLoads; ++u) {
          if (i + u >= m || from[i + u] < 0) continue;
          unsigned char* x = at(to[i + u]);
          if (c.vec == 16) *reinterpret_cast<uint4*>(x) = v[u];
          else *reinterpret_cast<uint32_t*>(x) = v[u].x;
        }
      }
    }
  }
}

template <typename... A>
cudaError_t launch(void (*kern)(A...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_copy_pages(const PagesParams& p, const int64_t* pairs, int64_t num_pairs, cudaStream_t stream) {
  const int64_t chunks = p.first_chunk[p.num_caches];
  const int64_t per_launch = 0x7fffffff / chunks;  // pairs that a grid holds
  for (int64_t first = 0; first < num_pairs; first += per_launch) {
    const int64_t n = num_pairs - first < per_launch ? num_pairs - first : per_launch;
    const cudaError_t e = launch<PagesParams, const int64_t*, int64_t>(copy_pages_kernel, dim3(unsigned(n * chunks)),
                                                                       kCopyThreads, stream, p, pairs, first);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_keep_tokens(const PagesParams& p, const KeepParams& k, cudaStream_t stream) {
  const dim3 grid(unsigned(k.num_seqs), unsigned(p.num_caches ? p.num_caches : 1));
  return launch<PagesParams, KeepParams>(keep_tokens_kernel, grid, kKeepThreads, stream, p, k);
}

}  // namespace pkv
