// tree_split.cuh — what the tensor-core attention kernels for drafted trees share: the split
// of the work over the blocks, bounded waits and copies, and the fold of split rows.
//
// An item is (sequence, KV head, item_nodes drafted nodes) and its work is its key tiles of
// 128 positions.  The items' work, laid end to end, is cut into equal contiguous ranges, one
// per block; an item cut by a border leaves a part per block, which the merge kernel folds.
#pragma once

#include <cuda.h>

#include "tree_common.cuh"

namespace pkv {
namespace tree {

constexpr int kBM = 128;  // rows per row tile
constexpr int kBN = 128;  // positions per key tile
constexpr float kGap = 8.f;  // growth of a row's maximum (log2) that moves its reference

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ bool test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done) : "r"(smem_addr(bar)), "r"(parity) : "memory");
  return done != 0;
}
// Bounded wait that gives up when another role of the block has (and tells them).  (Short: it
// is inlined wherever a role waits, and the roles' loops share the instruction caches.)
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint32_t polls = 0;
  bool ok;
  do {
    ok = mbar_try_wait(bar, parity);
  } while (!ok && ++polls < kWaitPolls && !*abort);
  if (!ok) *abort = 1;
  return ok;
}

// A sequence's work in tiles: key tiles x groups of nodes x KV heads.
struct SeqWork {
  Extent e;
  int base;    // first position of its first tile: the block that holds e.lo
  int tiles;   // key tiles of an item (at least one where there are rows)
  int pairs;   // groups of item_nodes nodes
  __device__ __forceinline__ void load(const TreeParams& p, const TreeSplit& sp, int s, bool* bad) {
    e = extent(p, s, bad);
    base = e.lo & ~(p.block_size - 1);
    tiles = max(1, (e.L - base + kBN - 1) / kBN);
    const uint32_t in = sp.item_nodes;
    pairs = e.n <= int(in) ? (e.n > 0) : int((uint32_t(e.n) + in - 1) / in);
  }
  __device__ __forceinline__ int row_tiles(const TreeSplit& sp, int pair) const {  // of group `pair`
    return min(sp.item_nodes, e.n - pair * sp.item_nodes) > sp.tq ? 2 : 1;
  }
  __device__ __forceinline__ int64_t items(const TreeParams& p) const {
    return int64_t(pairs) * p.num_kv_heads;  // (no rows: none)
  }
};

constexpr int kSeqs = 6;  // sequences of the range whose work is kept in shared memory

// A block's range of the work, in shared memory.
struct Range {
  int first_seq;             // the range's first sequence
  int cost;                  // units of an item beside its tiles
  int64_t first_off;         // the range's start in that sequence's work
  int64_t share, from, count;  // units of a block's range, where this one starts, what it holds
  SeqWork seqs[kSeqs];       // first_seq, first_seq + 1, ...
};

// Walks the item parts of a block's range; every role walks the same sequence.  The range
// is in units of work: an item is `cost` units for its start and end, then its tiles.
struct Walk {
  SeqWork q;
  int s, kvh, pair;
  int u0, u1;      // the part's units of the item
  int j0, j1;      // and its key tiles
  int nt;          // row tiles of the pair (1 or 2)
  int64_t left;    // units left in the range, this part's included
  __device__ __forceinline__ bool valid() const { return left > 0; }
  __device__ __forceinline__ bool begins() const { return j0 == 0; }
  __device__ __forceinline__ bool ends() const { return j1 == q.tiles; }
  // whether some position of tile j may be hidden from some row
  __device__ __forceinline__ bool cut(int j) const {
    const int pos = q.base + j * kBN;
    return pos + kBN > q.e.P || pos < q.e.lo;  // (P <= L)
  }
  __device__ __forceinline__ void part(const TreeSplit& sp, int cost) {
    u1 = int(min(int64_t(q.tiles + cost), u0 + left));
    j0 = max(0, u0 - cost);
    j1 = u1 - cost;
    if (j1 <= j0) left = 0;  // (the range ends before the item's first tile)
    nt = q.row_tiles(sp, pair);
  }
  __device__ __forceinline__ void load(const TreeParams& p, const TreeSplit& sp, const Range* rg) {
    const int i = s - rg->first_seq;
    bool bad;
    if (i < kSeqs) q = rg->seqs[i]; else q.load(p, sp, s, &bad);
  }
  __device__ __forceinline__ void start(const TreeParams& p, const TreeSplit& sp, const Range* rg) {
    left = rg->count;
    if (left <= 0) return;
    s = rg->first_seq;
    load(p, sp, rg);
    const int64_t off = rg->first_off;
    const uint32_t units = uint32_t(q.tiles + rg->cost);
    const int item = off < units ? 0 : off <= 0xffffffff ? int(uint32_t(off) / units) : int(off / units);
    u0 = int(off - int64_t(item) * units);
    kvh = q.pairs == 1 ? item : item / q.pairs;
    pair = item - kvh * q.pairs;
    part(sp, rg->cost);
  }
  __device__ __forceinline__ void next(const TreeParams& p, const TreeSplit& sp, const Range* rg) {
    left -= u1 - u0;
    if (left <= 0) return;
    u0 = 0;
    if (++pair == q.pairs) {
      pair = 0;
      if (++kvh == p.num_kv_heads) {
        kvh = 0;
        do {
          ++s;
          load(p, sp, rg);  // (units are left, so a later sequence has some)
        } while (q.pairs == 0 && s + 1 < p.num_seqs);
      }
    }
    part(sp, rg->cost);
  }
};

// Finds the block's range; all threads call it, and it ends with a barrier.  Returns whether
// some sequence of the batch has more than `few` nodes.  `warp_sum`: shared scratch, one entry
// per warp.
template <int kThreads>
__device__ __forceinline__ bool find_range(const TreeParams& p, const TreeSplit& sp, Range* rg, longlong2* warp_sum,
                                           int few) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // every thread adds up a run of sequences, then the one whose run holds the range's start
  // finds the sequence
  const int per = p.num_seqs <= kThreads ? 1 : (p.num_seqs + kThreads - 1) / kThreads;
  const int s0 = min(p.num_seqs, tid * per), s1 = min(p.num_seqs, s0 + per);
  SeqWork mine;  // the last one of the run (the only one where there are no more than threads)
  longlong2 sum = make_longlong2(0, 0);  // (tiles, items)
  bool many = false;
  for (int s = s0; s < s1; ++s) {
    bool bad;
    mine.load(p, sp, s, &bad);
    many |= mine.e.n > few;
    if (bad && blockIdx.x == 0) raise_device_error(p.err, kErrContextLen);
    sum.x += mine.tiles * mine.items(p);
    sum.y += mine.items(p);
  }
  longlong2 incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) {
      incl.x += x;
      incl.y += y;
    }
  }
  if (lane == 31) warp_sum[warp] = incl;
  many = __syncthreads_or(many);
  longlong2 before = make_longlong2(incl.x - sum.x, incl.y - sum.y), all = make_longlong2(0, 0);
  const int warps = (p.num_seqs + 32 * per - 1) / (32 * per);  // that hold sequences
  for (int w = 0; w < warps; ++w) {
    const longlong2 x = warp_sum[w];
    if (w < warp) {
      before.x += x.x;
      before.y += x.y;
    }
    all.x += x.x;
    all.y += x.y;
  }
  // an item's start and end take about as long as a tile; where a block has few tiles the
  // SMs matter more
  const int cost = all.x >= 4 * int64_t(gridDim.x) ? 1 : 0;
  const int64_t total = all.x + cost * all.y;
  const int64_t share = total <= 0x7fffffff ? int64_t((uint32_t(total) + gridDim.x - 1) / gridDim.x)
                                            : (total + gridDim.x - 1) / gridDim.x;
  const int64_t from = share * blockIdx.x, count = max(int64_t(0), min(share, total - from));
  int64_t at = before.x + cost * before.y;  // where this thread's run starts
  if (from >= at && from < at + sum.x + cost * sum.y) {
    for (int s = s0; s < s1; ++s) {
      SeqWork w = mine;
      bool bad;
      if (per > 1) w.load(p, sp, s, &bad);
      const int64_t n = (w.tiles + cost) * w.items(p);
      if (from < at + n) {
        rg->first_seq = s;
        rg->first_off = from - at;
        break;
      }
      at += n;
    }
  }
  if (tid == 0) {
    rg->cost = cost;
    rg->share = share;
    rg->from = from;
    rg->count = count;
  }
  __syncthreads();
  if (count > 0) {
    const int first = rg->first_seq;
    if (per == 1) {
      if (s0 < s1 && s0 >= first && s0 < first + kSeqs) rg->seqs[s0 - first] = mine;
    } else if (tid < kSeqs && first + tid < p.num_seqs) {
      SeqWork w;
      bool bad;
      w.load(p, sp, first + tid, &bad);
      rg->seqs[tid] = w;
    }
  }
  __syncthreads();
  return many;
}

// Folds the items cut by range borders.  Block (c, y): the item that begins in range c and
// goes on behind it, rows 32 y .. 32 y + 31 of its row tiles; a warp takes four of them at
// once (their loads overlap), its lanes D / 32 columns each.  The parts are taken in order.
// Bound by the latency of its loads: 6 us for 64 ragged sequences, most of it the launch.
constexpr int kMergeWarps = 8, kMergeRows = 32;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const __grid_constant__ TreeParams p, const TreeSplit sp) {
  // (no early launch of the next kernel: one block of the next call's main kernel on an SM
  // keeps this kernel's blocks off it, 72 -> 106 us per call on ragged trees back to back)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kCols = D / 32, kRows = kMergeRows / kMergeWarps;
  const int c = int(blockIdx.x);
  const TreeSplit::Tail t = sp.tails[c];
  const int g = p.group, TQ = sp.tq;
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  int row[kRows], node[kRows];
  bool live[kRows], any = false;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    row[i] = int(blockIdx.y) * kMergeRows + i * kMergeWarps + warp;
    const int qt = row[i] / kBM, r = row[i] % kBM;
    node[i] = qt * TQ + r / g;
    live[i] = r < TQ * g && node[i] < t.nodes;
    any |= live[i];
  }
  if (!any) return;
  float M[kRows], den[kRows], o[kRows][kCols];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    M[i] = -INFINITY;
    den[i] = 0.f;
#pragma unroll
    for (int k = 0; k < kCols; ++k) o[i][k] = 0.f;
  }
  constexpr int kInFlight = 2;
  for (int b0 = c; b0 <= t.last; b0 += kInFlight) {
    float2 ml[kInFlight][kRows];
    float v[kInFlight][kRows][kCols];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        ml[u][i] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int k = 0; k < kCols; ++k) v[u][i][k] = 0.f;
        if (b0 + u <= t.last && live[i]) {
          const int64_t pr = int64_t(2 * (b0 + u) + (b0 + u == c ? 1 : 0)) * sp.rows + row[i];
          ml[u][i] = sp.ml[pr];
          const float* src = sp.o + pr * D + lane * kCols;
          if constexpr (kCols == 4) {
            const float4 f = *reinterpret_cast<const float4*>(src);
            v[u][i][0] = f.x; v[u][i][1] = f.y; v[u][i][2] = f.z; v[u][i][3] = f.w;
          } else {
            const float2 f = *reinterpret_cast<const float2*>(src);
            v[u][i][0] = f.x; v[u][i][1] = f.y;
          }
        }
      }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        // (a part whose positions the row does not see, or whose scores are all NaN, has no
        // maximum: it counts as it stands)
        const float m2 = fmaxf(M[i], ml[u][i].x), ref = m2 == -INFINITY ? 0.f : m2;
        const float a = M[i] == -INFINITY ? 1.f : fast_exp2(M[i] - ref);
        const float b = ml[u][i].x == -INFINITY ? 1.f : fast_exp2(ml[u][i].x - ref);
        den[i] = den[i] * a + ml[u][i].y * b;
#pragma unroll
        for (int k = 0; k < kCols; ++k) o[i][k] = o[i][k] * a + v[u][i][k] * b;
        M[i] = m2;
      }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (!live[i]) continue;
    const float inv = den[i] != 0.f ? 1.f / den[i] : 0.f;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + int64_t(t.row0 + node[i]) * p.out_stride_t +
                         int64_t(t.kvh * g + (row[i] % kBM) % g) * p.out_stride_h + lane * kCols;
#pragma unroll
    for (int k = 0; k < kCols; k += 2) {
      const __nv_bfloat162 pr = __floats2bfloat162_rn(o[i][k] * inv, o[i][k + 1] * inv);
      if (sp.out_vec) {
        *reinterpret_cast<uint32_t*>(out + k) = *reinterpret_cast<const uint32_t*>(&pr);
      } else {  // (rows at any address)
        out[k] = pr.x;
        out[k + 1] = pr.y;
      }
    }
  }
}

}  // namespace tree
}  // namespace pkv
