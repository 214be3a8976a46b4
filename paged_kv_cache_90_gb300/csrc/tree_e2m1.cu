// tree_e2m1.cu — attention of drafted trees (and decode of more than 16 heads a KV head, or over
// blocks of 2 and 4 tokens) over a 4-bit cache on the fifth-generation tensor cores.
//
// A row tile is 128 MMA rows: a KV head's g query heads times up to TQ = 128 / g drafted nodes; an
// item is (sequence, KV head, one or two row tiles) and its work is its key tiles of 128 positions,
// cut into equal ranges as in tree_split.cuh.  A step is one (key tile, row tile):
//   S = Q K^T          M 128, N 128, K = D: both f16 in shared memory (128-byte swizzle), S in one
//                      of two tensor-memory buffers, by the step's parity
//   P = 2^(S c - m)    written back over S as f16 pairs by a softmax warpgroup, a row per thread
//   O += P V           M 128, N = D, K = 128 keys: P from tensor memory, V from shared memory
// Two softmax warpgroups work on an item, each with a reference m, a sum and an O of its own: two row
// tiles go to one each; of a single one each has half the keys of every tile, and their two results
// are folded when the item ends (each then writes half of the columns).  A step of one row tile is
// then half as long in a warpgroup, and so is the chain from its scores to its product.
//
// K and V are widened by a warpgroup each: a warp loads 32 positions of a tile into registers, a tile
// ahead, and code times group scale is an f16 number exactly (e2m1_codes.cuh).  (With asynchronous
// copies into shared memory a warp spent 500 clocks a tile on issuing them and 150 on reading them.)
// A query row is scaled by the power of two that brings its largest element to 2^14, so its bf16
// values are exact down to 2^-29 of that.  A weight is rounded to f16, half a step, 2^-11, down to
// 2^-21 of the row's largest, 2^-32 of that below.  Scores, maximum, sum and output are binary32.
//
// 32 trees of 8 to 32 nodes over 1000 to 8192 positions, 32 : 8 heads of 128 (182 MB): 108 us; on the
// CUDA cores 8 ms.  Neither memory (21 % of the time) nor the tensor cores (36 %) bound it but a tile's
// chain: about 2700 clocks of products (1240), weights (1024 of the exponentials) and widening, of
// which two tiles' buffers hide no more than a part.  Without the softmax it takes 86 us, without the
// widening 95, with a single product a step 71.  Two warpgroups on one row tile's keys took 120 us
// down to 108.  Tried without gain: a second MMA warp (114 us), a half tile's scores kept in
// registers between maximum and weights (110) and S given back as soon as they are there (116), waits
// that spin (129), one lane that waits for its warp (113), a step's waits at once (110), four MMAs an
// election (110).  The MMA warp's own way through a tile, 2000 to 2500 clocks between the other roles'
// instructions, is what the others wait for.
//
// Nothing that a row does not see reaches it: hidden scores become -infinity, V rows outside the
// context are widened as zeros, and so are groups of drafted nodes whose scale is a NaN: the rows
// that see such a node get the NaN back with their output.
//
// Warps: 1 issues the MMAs; 4-7 and 8-11 are the softmax warpgroups, which also convert the queries;
// 12-15 widen K, 16-19 V.  Every wait is bounded; when one runs out the block sets an
// error bit and a flag that makes every role stop, lets its copies and MMAs land and frees the
// tensor memory.
#include <algorithm>
#include <mutex>

#include "e2m1_codes.cuh"
#include "f32x2.cuh"
#include "i8_codes.cuh"
#include "tcgen05.cuh"
#include "tree_split.cuh"
#include "umma.cuh"

namespace pkv {
namespace tree_e2m1 {

using namespace tree;

constexpr int kThreads = 640;
// registers of a thread, by warpgroup: launched with 96 each (5 x 96 = 480), then split anew
constexpr int kRegsControl = 40, kRegsSoftmax = 136, kRegsWiden = 80;
static_assert(kRegsControl + 2 * kRegsSoftmax + 2 * kRegsWiden <= 5 * 96, "registers");
constexpr uint32_t kTmemCols = 512;
// A row's weights are 2^(z - m + kTop): at most 2^15 with a reference that lags by 2^kGap.
constexpr float kTop = 7.f;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;             // 64-column halves of an operand (128-byte rows)
  static constexpr uint32_t kHalfBytes = kBM * 128;  // 16 KB
  static constexpr uint32_t kOpBytes = kHalves * kHalfBytes;
  static constexpr int kRow = D / 2, kGroups = D / 16;  // bytes and scales of a cache row
  // from the 1024-aligned base: two query tiles | two K tiles | two V tiles | state
  static constexpr uint32_t kQ = 0, kK = 2 * kOpBytes, kV = 4 * kOpBytes, kState = 6 * kOpBytes;
  static constexpr uint32_t kStateBytes = 11 * 1024;
  static constexpr size_t kSmem = kState + kStateBytes + 1024;  // (+ alignment)
  // tensor memory: S of even and odd steps (128 columns each), then O of the two warpgroups
  static constexpr uint32_t kS = 0, kO = 2 * kBN;
};

// Barriers.  A wait names a phase by its parity, so its barrier may be at most one phase away:
// those that a softmax warpgroup waits for count its own steps, two barriers by their parity.
enum Bar { kQFull = 0, kQEmpty = 2, kKFull = 4, kKEmpty = 6, kVFull = 8, kVEmpty = 10, kSFull = 12, kPFull = 16,
           kODone = 20, kOFree = 24, kStat = 25, kDrain = 27, kNumBars = 28 };

constexpr int kQueryTiles = 4;  // row tiles whose score factors are kept: those of two items
constexpr int kBadItems = 8;    // items whose bad rows are kept: the widening is up to three ahead

struct State {
  uint64_t bars[kNumBars];
  volatile int abort;
  uint32_t tmem;
  Range range;
  longlong2 warp_sum[kThreads / 32];
  float qf[kQueryTiles][kBM];     // a row's score factor
  float2 stat[2][2][kBM];         // a warpgroup's maximum and sum of a row at an item's end
  // drafted positions with a NaN scale in V, 8 to a byte from the first tile that holds drafted
  // nodes on (1024 nodes touch at most 9 tiles)
  unsigned char bad[kBadItems][144];
  // What a widening warp of V has to know of an item's part (mod 8: its walk is up to three tiles, so
  // items, ahead): tiles, the first one's first position, the context's end, its window's start and
  // its drafted nodes', and the first tile of these counted from the part's first.
  struct Item {
    int tiles, pos, L, lo, P, jt;
  } item[4][8];
};

__device__ __forceinline__ bool wait(State* st, int bar, uint32_t parity) {
  return tree::wait(&st->bars[bar], parity, &st->abort);
}
__device__ __forceinline__ bool wait_warp(State* st, int bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(st, bar, parity));
}

// a lane's D / 4 codes of a row, and their scales (two, or one at D = 64)
__device__ __forceinline__ void load_codes(const unsigned char* p, uint32_t (&w)[4]) {
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
}
__device__ __forceinline__ void load_codes(const unsigned char* p, uint32_t (&w)[2]) {
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
}
template <int D>
__device__ __forceinline__ uint32_t load_scales(const unsigned char* p) {
  uint32_t x;
  if (D == 128) asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(x) : "l"(p));
  else asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

template <int N>
__device__ __forceinline__ void less_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// f16 x f16 -> f32, M x N, A and B K-major (0) or MN-major (1)
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// The positions pos .. pos + 127 of a tile that a row sees, 64 to a word.
__device__ __forceinline__ void tile_bits(const Extent& e, int pos, const int64_t* mask, uint64_t word0, uint64_t (&k)[2]) {
  auto ones = [](int n) -> uint64_t { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; };
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int p0 = pos + 64 * w;
    uint64_t b = ones(e.P - p0) & ~ones(e.lo - p0);  // (before the nodes; with no mask P is the end)
    if (mask) {
      // bit i is node c + i
      const int c = p0 - e.P;
      if (c < e.n && c > -64) {
        uint64_t m;
        if (c < 0) {
          m = word0 << -c;
        } else {
          const int i = c >> 6, o = c & 63;
          m = (i == 0 ? word0 : uint64_t(__ldg(mask + i))) >> o;
          if (o && 64 * (i + 1) < e.n) m |= uint64_t(__ldg(mask + i + 1)) << (64 - o);
        }
        b |= m & ones(e.L - p0) & ~ones(e.P - p0);
      }
    }
    k[w] = b;
  }
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// Largest of a row's 32 scores at tensor-memory column `ts`; with kCut those not kept become
// -infinity there.
template <bool kCut>
__device__ __forceinline__ float row_max(uint32_t ts, uint32_t keep) {
  uint32_t w[32];
  tc::ld32(ts, w);
  tc::wait_ld();
  if (kCut) {
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = keep >> i & 1u ? w[i] : 0xff800000u;
    tc::st32(ts, w);
  }
  float t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = max3(__uint_as_float(w[i]), __uint_as_float(w[4 + i]), __uint_as_float(w[8 + i]));
#pragma unroll
  for (int i = 12; i < 28; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = max3(t[k], __uint_as_float(w[i + k]), __uint_as_float(w[i + 4 + k]));
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = fmaxf(t[i], __uint_as_float(w[28 + i]));
  return max3(fmaxf(t[0], t[1]), t[2], t[3]);
}

// Weights 2^(score * sl - mu) of a row's 32 scores at column `ts`, written as f16 pairs to column
// `tp` (whose scores have been read); returns their sum.
__device__ __forceinline__ float weights(uint32_t ts, uint32_t tp, float sl, float mu) {
  uint32_t w[32], pk[16];
  tc::ld32(ts, w);
  tc::wait_ld();
  const uint64_t sl2 = pack2(sl, sl), mu2 = pack2(-mu, -mu);
  uint64_t ps[2] = {0ull, 0ull};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 z = unpack2(fma2(pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), sl2, mu2));
    const float a = fast_exp2(z.x), b = fast_exp2(z.y);
    ps[i & 1] = add2(ps[i & 1], pack2(a, b));
    const __half2 pr = __floats2half2_rn(a, b);
    pk[i] = *reinterpret_cast<const uint32_t*>(&pr);
  }
  tc::st16(tp, pk);
  const float2 sum = unpack2(add2(ps[0], ps[1]));
  return sum.x + sum.y;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tree_e2m1_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeSplit sp) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  State* st = reinterpret_cast<State*>(smem + C::kState);
  // (the warp's number from one lane: the compiler then knows that it is the same in all)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int g = p.group, TQ = sp.tq;
  const uint32_t sbase = smem_addr(smem);

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      // one arrival a warp where warps arrive
      const bool warps4 = (i >= kKFull && i < kKFull + 2) || (i >= kVFull && i < kVFull + 2) ||
                          (i >= kPFull && i < kPFull + 4) || (i >= kStat && i < kStat + 2);
      const bool warps8 = i == kOFree || (i >= kQFull && i < kQFull + 2);
      mbar_init(&st->bars[i], warps8 ? 8 : warps4 ? 4 : 1);
    }
    st->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) tc::alloc(&st->tmem, kTmemCols);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing of the caller's is read before
  asm volatile("griddepcontrol.launch_dependents;");
  (void)find_range<kThreads>(p, sp, &st->range, st->warp_sum, 0);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = st->tmem;
  const Range* rg = &st->range;

  // (a warpgroup takes its registers together, by one instruction, and its roles part behind it)
  if (warp < 4) {
    less_registers<kRegsControl>();
    if (warp == 1) {
      Walk it;
      it.start(p, sp, rg);
      // ---- MMAs (a warp, see umma.cuh): S of a step, then P V of the step before it -------------------
      // (Counters and descriptors come from values that the compiler knows to be the warp's: a lane's
      // own would be moved to uniform registers for every MMA.)
      constexpr uint32_t idS = idesc_f16(kBM, kBN, 0, 0), idO = idesc_f16(kBM, D, 0, 1);
      constexpr uint64_t kOp = C::kOpBytes >> 4, kHalf = C::kHalfBytes >> 4;  // (descriptors hold addresses / 16)
      auto one = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      const uint32_t base = one(int(sbase)), tm = one(int(tmem));
      const uint64_t qdesc = tc::desc_sw128(base + C::kQ, 16, 1024), kdesc = tc::desc_sw128(base + C::kK, 16, 1024);
      const uint64_t vdesc = tc::desc_sw128(base + C::kV, C::kHalfBytes, 1024);
      int xs = 0, tiles = 0, q = 0, item = 0, steps[2] = {0, 0};  // (steps: of the warpgroups)
      // the step whose P V is next: its tile, and what it is to the one warpgroup that has it, or to both
      // (-1); whether it is its warpgroup's first of the item, and the last of its tile
      int p_wg = 0, p_step[2] = {0, 0}, p_tile = 0, p_item = 0;
      bool p_first = false, p_last = false, p_due = false, ok = true;
      auto products = [&]() {
        const int x = xs - 1;
        const uint64_t vd = vdesc + (p_tile & 1) * kOp;
        const uint32_t ts = tm + C::kS + (x & 1) * kBN;
        ok = wait_warp(st, kVFull + (p_tile & 1), uint32_t(p_tile >> 1) & 1u) &&
             (!p_first || p_item == 0 || wait_warp(st, kOFree, uint32_t(p_item - 1) & 1u));
        if (p_wg >= 0) {
          const int w = p_wg, n = w ? p_step[1] : p_step[0];
          ok = ok && wait_warp(st, kPFull + 2 * w + (n & 1), uint32_t(n >> 1) & 1u);
          if (!ok) return;
          tc::fence_after();
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            umma::mma_ts(tm + C::kO + w * D, ts + 8 * kk, vd + kk * (16 * 128 >> 4), idO, (!p_first || kk > 0) ? 1u : 0u);
          umma::commit(&st->bars[kODone + 2 * w + (n & 1)]);
        } else {
#pragma unroll
          for (int w = 0; w < 2; ++w) {  // a half of the keys each
            const int n = p_step[w];
            ok = ok && wait_warp(st, kPFull + 2 * w + (n & 1), uint32_t(n >> 1) & 1u);
            if (!ok) return;
            tc::fence_after();
#pragma unroll
            for (int kk = 0; kk < kBN / 32; ++kk)
              umma::mma_ts(tm + C::kO + w * D, ts + 64 * w + 8 * kk, vd + (4 * w + kk) * (16 * 128 >> 4), idO,
                           (!p_first || kk > 0) ? 1u : 0u);
            umma::commit(&st->bars[kODone + 2 * w + (n & 1)]);
          }
        }
        if (p_last) umma::commit(&st->bars[kVEmpty + (p_tile & 1)]);
        p_due = false;
      };
      for (; ok && it.valid(); it.next(p, sp, rg), ++item) {
        const int nt = one(it.nt), count = one(it.j1 - it.j0) * nt;
        for (int i = 0; ok && i < count; ++i) {
          const int qt = nt == 2 ? i & 1 : 0, qs = (q + qt) & 1, use = (q + qt) >> 1;
          // (an item's queries may be late: the products do not wait for them)
          if (i == 0 && p_due && !__all_sync(0xffffffffu, test_wait(&st->bars[kQFull + qs], uint32_t(use) & 1u))) products();
          if (qt == 0) ok = ok && wait_warp(st, kKFull + (tiles & 1), uint32_t(tiles >> 1) & 1u);
          if (i < nt) ok = ok && wait_warp(st, kQFull + qs, uint32_t(use) & 1u);
          if (!ok) break;
          tc::fence_after();
          const uint64_t qd = qdesc + qs * kOp, kd = kdesc + (tiles & 1) * kOp;
          const uint32_t ts = tm + C::kS + (xs & 1) * kBN;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma::mma_ss(ts, qd + (kk >> 2) * kHalf + (kk & 3) * 2, kd + (kk >> 2) * kHalf + (kk & 3) * 2, idS, kk > 0 ? 1u : 0u);
          if (nt == 1 || qt == 0) umma::commit(&st->bars[kSFull + (steps[0] & 1)]);
          if (nt == 1 || qt == 1) umma::commit(&st->bars[kSFull + 2 + (steps[1] & 1)]);
          if (qt == nt - 1) umma::commit(&st->bars[kKEmpty + (tiles & 1)]);
          if (i >= count - nt) umma::commit(&st->bars[kQEmpty + qs]);
          if (p_due) products();
          p_due = true;
          p_wg = nt == 1 ? -1 : qt;
          p_step[0] = steps[0];
          p_step[1] = steps[1];
          p_tile = tiles;
          p_item = item;
          p_first = i < nt;
          p_last = qt == nt - 1;
          ++xs;
          if (nt == 1 || qt == 0) ++steps[0];
          if (nt == 1 || qt == 1) ++steps[1];
          if (qt == nt - 1) ++tiles;
        }
        q += nt;
      }
      if (ok && p_due) products();
      // every MMA issued has completed before the tensor memory is freed
      umma::commit(&st->bars[kDrain]);
      (void)mbar_wait_bounded(&st->bars[kDrain], 0);
      if (!ok) {
        st->abort = 1;
        if (lane == 0) raise_device_error(p.err, kErrTimeout);
      }
    } else if (warp == 0) {
      // ---- what the fold needs of an item that goes on in the next block's range ----------------------
      Walk it;
      int64_t at = rg->from;
      TreeSplit::Tail tail = {0, 0, 0, 0};
      for (it.start(p, sp, rg); it.valid(); it.next(p, sp, rg)) {
        if (it.begins() && !it.ends()) {
          const int node0 = 2 * it.pair * TQ;
          tail.row0 = it.q.e.q0 + node0;
          tail.nodes = min(2 * TQ, it.q.e.n - node0);
          tail.kvh = it.kvh;
          tail.last = int((at - it.u0 + it.q.tiles + rg->cost - 1) / rg->share);
        }
        at += it.u1 - it.u0;
      }
      if (lane == 0) sp.tails[blockIdx.x] = tail;
    }
  } else if (warp >= 12) {
    less_registers<kRegsWiden>();
    Walk it;
    it.start(p, sp, rg);
    // ---- widening: K by one warpgroup, V by the other; a warp has 32 positions of every tile --------
    const bool isv = warp >= 16;
    const int w4 = warp & 3, gr = lane >> 2, t = lane & 3;  // (D = 128: a lane has 16 bytes of a row)
    const int bs_mask = p.block_size - 1;
    const uint64_t block_bytes = uint32_t(p.cs_block), block_scales = uint32_t(p.ts_block);  // (32 bits: see the host's check)
    const uint64_t head_bytes = uint32_t(p.cs_head), head_scales = uint32_t(p.ts_head);
    unsigned char* const tiles = smem + (isv ? C::kV : C::kK);
    constexpr int kW = D / 32, kN = 32 / 8;  // words of a lane, its rows
    // (a tile's first position is a block's first.)  The lanes of a row's second half take their words in
    // another order, so that eight lanes never meet a bank twice when they write them.
    const unsigned char* const cache = static_cast<const unsigned char*>(isv ? p.value_cache : p.key_cache) + 4 * kW * t;
    const unsigned char* const scales = (isv ? p.v_group_scales : p.k_group_scales) + (D / 64) * t;
    // the table's entries are looked up a tile ahead of the loads; the walk is theirs, an item ahead
    int items = 0, t_left = 0, t_pos = 0, t_end = 0, next_kvh = 0;
    const int32_t* t_entry = nullptr;
    bool have_next = false;
    uint32_t e_next = 0;
    auto lookup = [&]() {
      if (t_left == 0) {
        have_next = it.valid();
        if (!have_next) return;
        t_left = it.j1 - it.j0;
        const int pos0 = it.q.base + it.j0 * kBN + 32 * w4;
        t_pos = pos0 + lane;
        t_end = it.q.e.L;
        t_entry = p.block_tables + int64_t(it.s) * p.bt_stride + (t_pos >> sp.bs_shift);
        next_kvh = it.kvh;
        if (isv && lane == 0)
          st->item[w4][items & 7] = {t_left, pos0, it.q.e.L, it.q.e.lo, it.q.e.P, (it.q.e.P - it.q.base) / kBN - it.j0};
        __syncwarp();  // (the other lanes read it later)
        ++items;
        it.next(p, sp, rg);
      }
      // (positions behind the context are read from block 0, whose numbers have no part)
      e_next = t_pos < t_end ? uint32_t(__ldg(t_entry)) : 0u;
      t_pos += kBN;
      t_entry += kBN >> sp.bs_shift;
      --t_left;
    };
    auto load = [&](uint32_t (&x)[kN][kW], uint32_t (&sc)[kN]) {
      uint32_t e = e_next;
      if (e >= uint32_t(p.num_blocks)) {  // (negative ones are large)
        raise_device_error(p.err, kErrTableEntry);
        e = 0;
      }
      uint32_t blk[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) blk[i] = __shfl_sync(0xffffffffu, e, 8 * i + gr);
      const unsigned char *const from = cache + next_kvh * head_bytes, *const sfrom = scales + next_kvh * head_scales;
#pragma unroll
      for (int i = 0; i < kN; ++i) load_codes(from + blk[i] * block_bytes + ((8 * i + gr) & bs_mask) * C::kRow, x[i]);
#pragma unroll
      for (int i = 0; i < kN; ++i)
        sc[i] = load_scales<D>(sfrom + blk[i] * block_scales + ((8 * i + gr) & bs_mask) * C::kGroups);
      lookup();
    };
    lookup();
    bool have = have_next, ok = true;
    uint32_t x[kN][kW], sc[kN];
    if (have) load(x, sc);
    State::Item part = {};  // the tile's, and how many of its tiles are left
    int item = 0, k_tile = 0;
    for (int n = 0; have; ++n) {
      const bool more = have_next;
      uint32_t y[kN][kW], sy[kN];
      if (more) load(y, sy);
      if (isv) {
        if (k_tile == part.tiles) {
          part = st->item[w4][item & 7];
          ++item;
          k_tile = 0;
        }
        if (part.pos - 32 * w4 + kBN > part.P || part.pos - 32 * w4 < part.lo) {  // (Walk::cut)
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const int pos = part.pos + 8 * i + gr;
            bool bad = false;
            if (pos >= part.L || pos < part.lo) {
              sc[i] = 0;
            } else if (pos >= part.P) {
              if ((sc[i] & 0x7fu) == 0x7fu) { sc[i] &= 0xff00u; bad = true; }
              if ((sc[i] & 0x7f00u) == 0x7f00u) { sc[i] &= 0xffu; bad = true; }
            }
            uint32_t m = __ballot_sync(0xffffffffu, bad), byte = 0;
            if (m) {
#pragma unroll
              for (int k = 0; k < 8; ++k) byte |= (m >> (4 * k) & 15u) ? 1u << k : 0u;
            }
            if (lane == 0 && k_tile >= part.jt)
              st->bad[(item - 1) % kBadItems][16 * (k_tile - part.jt) + 4 * w4 + i] = static_cast<unsigned char>(byte);
          }
        }
        part.pos += kBN;
        ++k_tile;
      }
      const int buf = n & 1;
      if (n > 1 && !(ok = wait_warp(st, (isv ? kVEmpty : kKEmpty) + buf, uint32_t((n >> 1) - 1) & 1u))) break;
      const bool swap = D == 128 && t >= 2;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t two = e2m1::scales2(sc[i]);
        // (a word is half a group: two of the lane's first group, then of its second, or the other way round)
        const uint32_t in_order = swap ? __byte_perm(two, two, 0x1032) : two;
        const __half2 gs = *reinterpret_cast<const __half2*>(&in_order);
        const int row = 32 * w4 + 8 * i + gr;
        unsigned char* to = tiles + buf * C::kOpBytes + (D == 128 ? (t >> 1) * C::kHalfBytes : 0) + row * 128;
        const int cell0 = D == 128 ? (4 * (t & 1)) ^ (t & 2) : 2 * t;  // (with c, the order in which the words come)
#pragma unroll
        for (int c = 0; c < kW; ++c) {
          const __half2 s = c < 2 ? __low2half2(gs) : __high2half2(gs);
          uint32_t h[4];
          e2m1::widen8(D == 128 && swap ? x[i][(c ^ 2) % kW] : x[i][c], h);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[u]), s);
            h[u] = *reinterpret_cast<const uint32_t*>(&v);
          }
          *reinterpret_cast<uint4*>(to + ((cell0 ^ c ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&st->bars[(isv ? kVFull : kKFull) + buf]);
      have = more;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        sc[i] = sy[i];
#pragma unroll
        for (int c = 0; c < kW; ++c) x[i][c] = y[i][c];
      }
    }
    if (!ok && lane == 0) {
      st->abort = 1;
      raise_device_error(p.err, kErrTimeout);
    }
  } else {
    more_registers<kRegsSoftmax>();
    Walk it;
    it.start(p, sp, rg);
    // ---- softmax warpgroup `wg`: row r of its row tiles, r = tensor-memory lane ---------------------
    const int wg = (warp >> 2) - 1, q = warp & 3;
    const int r = 32 * q + lane, r_node = r / g, r_head = r - r_node * g;
    const uint32_t lane_off = uint32_t(32 * q) << 16;
    const uint32_t tO = tmem + C::kO + wg * D + lane_off;
    int x0 = 0, qc = 0, item = 0, steps = 0, folds = 0;  // `steps`: of this warpgroup so far; `folds`: items of one row tile
    bool ok = true;
    // The walk's item's queries: a row tile by each warpgroup, or half the rows of one by each.  They
    // are converted to f16, every row scaled by a power of two of its own.  (Between two items, before
    // the first one's output: the next one's scores are then under way.)
    auto queries = [&]() {
      constexpr int kLanes = D / 8, kPer = 32 / kLanes, kBatch = 4;  // lanes of a row, rows of a pass, passes
      const int sub = lane / kLanes, col = (lane % kLanes) * 8;
      const int qt = it.nt == 2 ? wg : 0, n = qc + qt, qs = n & 1, use = n >> 1;
      const int node0 = (2 * it.pair + qt) * TQ, rows = min(TQ, it.q.e.n - node0) * g;
      const float f = p.qk_scale_log2 * (p.k_head_scales ? __ldg(p.k_head_scales + it.kvh) : 1.f);
      if (use > 0) ok = ok && wait_warp(st, kQEmpty + qs, uint32_t(use - 1) & 1u);
      unsigned char* to = smem + C::kQ + qs * C::kOpBytes;
      const int w = it.nt == 2 ? q : 4 * wg + q, warps = it.nt == 2 ? 4 : 8;
      if (ok) {
#pragma unroll 1
        for (int r0 = w * kBatch * kPer; r0 < rows; r0 += warps * kBatch * kPer) {
          uint4 x[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int r = r0 + u * kPer + sub;
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows) {
              const int node = r / g, h = r - node * g;
              x[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.query) +
                                                     int64_t(it.q.e.q0 + node0 + node) * p.q_stride_t +
                                                     int64_t(it.kvh * g + h) * p.q_stride_h + col);
            }
          }
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int r = r0 + u * kPer + sub;
            float y[8], top = 0.f;
            Chunk<BF16>::expand(x[u], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int sh = i8::query_shift(top);
            const float s = copysignf(i8::power(sh), f);  // (the factor is positive: a row's maximum is that of its sums)
            if (r < rows) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __half2 v = __floats2half2_rn(y[2 * e] * s, y[2 * e + 1] * s);
                h[e] = *reinterpret_cast<const uint32_t*>(&v);
              }
              *reinterpret_cast<uint4*>(to + (col >> 6) * C::kHalfBytes + r * 128 + (((col >> 3) & 7) ^ (r & 7)) * 16) =
                  make_uint4(h[0], h[1], h[2], h[3]);
              // (never 0, with which a hidden score of -infinity would be NaN)
              const float factor = fabsf(f) * i8::power(-sh);
              if (col == 0) st->qf[n % kQueryTiles][r] = factor < 0x1p-149f ? 0x1p-149f : factor;
            }
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&st->bars[kQFull + qs]);
        if (it.nt == 2) mbar_arrive(&st->bars[kQFull + qs]);  // (eight arrivals, whoever makes them)
      }
    };
    if (it.valid()) queries();
    for (; ok && it.valid(); ++item) {
      const Extent e = it.q.e;
      const int total = (it.j1 - it.j0) * it.nt, qt = it.nt == 2 ? wg : 0;
      const int node = (2 * it.pair + qt) * TQ + r_node;
      const bool row_ok = r < TQ * g && node < e.n;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      const int64_t trow = int64_t(e.q0) + node;
      const int64_t* mask = p.tree_mask ? p.tree_mask + (row_ok ? trow : int64_t(e.q0)) * p.mask_stride : nullptr;  // (idle rows: any)
      const uint64_t word0 = mask ? uint64_t(__ldg(mask)) : 0;
      float m_ref = -INFINITY, l_run = 0.f, sl = 0.f;
      // this warpgroup's part of a step: its columns of S, 32 at a time
      const int half = it.nt == 1 ? wg : 0, chunks = it.nt == 1 ? 2 : 4;
      for (int j = it.j0; j < it.j1; ++j, ++steps) {
        const int x = x0 + (j - it.j0) * it.nt + qt;
        const int pos = it.q.base + j * kBN;
        const uint32_t tS = tmem + C::kS + (x & 1) * kBN + 64 * half + lane_off;
        if (!(ok = wait_warp(st, kSFull + 2 * wg + (steps & 1), uint32_t(steps >> 1) & 1u))) break;
        tc::fence_after();
        if (warp_ok) {
          if (j == it.j0) sl = st->qf[(qc + qt) % kQueryTiles][r];
          float mx = -INFINITY;
          if (it.cut(j)) {
            uint64_t k[2];
            tile_bits(e, pos, mask, word0, k);
            if (half) k[0] = k[1];
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              mx = fmaxf(mx, row_max<true>(tS + 32 * c, uint32_t(k[0])));
              k[0] = k[0] >> 32 | k[1] << 32;
              k[1] >>= 32;
            }
            tc::wait_st();
          } else {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) mx = fmaxf(mx, row_max<false>(tS + 32 * c, 0u));
          }
          mx *= sl;
          const bool first = m_ref == -INFINITY;
          const bool move = row_ok && mx != -INFINITY && (first || mx > m_ref + kGap);
          if (__any_sync(0xffffffffu, move && !first)) {
            // some row's O is rescaled: its product of the step before has to be in it
            if (!(ok = wait_warp(st, kODone + 2 * wg + ((steps - 1) & 1), uint32_t((steps - 1) >> 1) & 1u))) break;
            tc::fence_after();
            const float alpha = move && !first ? fast_exp2(m_ref - mx) : 1.f;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t w[32];
              tc::ld32(tO + 32 * c, w);
              tc::wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * alpha);
              tc::st32(tO + 32 * c, w);
            }
            tc::wait_st();
            l_run *= alpha;
          }
          if (move) m_ref = mx;
          const float mu = m_ref == -INFINITY ? 0.f : m_ref - kTop;
          float sum = 0.f;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) sum += weights(tS + 32 * c, tS + 16 * c, sl, mu);
          l_run += sum;
          tc::wait_st();
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->bars[kPFull + 2 * wg + (steps & 1)]);
      }
      if (!ok) break;
      x0 += total;
      qc += it.nt;
      // (what the output needs of the walk, which goes on to the next item's queries)
      const int nt = it.nt, j0 = it.j0, j1 = it.j1, base = it.q.base, kvh = it.kvh;
      const bool begins = it.begins(), whole = begins && it.ends();
      const int32_t* const table = p.block_tables + int64_t(it.s) * p.bt_stride;
      it.next(p, sp, rg);
      if (it.valid()) queries();
      if (!ok) break;
      // ---- the part's output: this warpgroup's row tile, or half the columns of both results ---------
      if (!(ok = wait_warp(st, kODone + 2 * wg + ((steps - 1) & 1), uint32_t((steps - 1) >> 1) & 1u))) break;
      float f0 = 1.f, f1 = 0.f, m = m_ref, l = l_run;  // the factors on this warpgroup's O and on the other's
      if (nt == 1) {
        st->stat[folds & 1][wg][r] = make_float2(m_ref, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->bars[kStat + wg]);
        if (!(ok = wait_warp(st, kStat + (wg ^ 1), uint32_t(folds) & 1u))) break;
        const float2 o = st->stat[folds & 1][wg ^ 1][r];
        ++folds;
        m = fmaxf(m_ref, o.x);
        const float ref = m == -INFINITY ? 0.f : m;
        // (rows whose scores are all NaN have no maximum: they count as they stand)
        f0 = m_ref == -INFINITY ? 1.f : fast_exp2(m_ref - ref);
        f1 = o.x == -INFINITY ? 1.f : fast_exp2(o.x - ref);
        l = wg ? o.y * f1 + l_run * f0 : l_run * f0 + o.y * f1;
      }
      tc::fence_after();
      if (warp_ok) {
        const float fv = p.v_head_scales ? __ldg(p.v_head_scales + kvh) : p.v_scale;
        const float inv = (whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f) * fv;
        const int64_t prow = int64_t(2 * blockIdx.x + (begins ? 1 : 0)) * sp.rows + qt * kBM + r;
        if (row_ok && !whole && (nt == 2 || wg == 0)) sp.ml[prow] = make_float2(m, l);
        const int jt = (e.P - base) / kBN;
        // (the bytes of this part's tiles; the others are not this item's)
        const unsigned char* bad = st->bad[item % kBadItems];
        const int b0 = 16 * (max(j0, jt) - jt), b1 = 16 * (j1 - jt);
        bool any_bad = false;
        if (mask && row_ok)
          for (int b = b0; b < b1; b += 4) any_bad |= *reinterpret_cast<const uint32_t*>(bad + b) != 0u;
        const int c_first = nt == 2 ? 0 : wg * (D / 64), c_last = nt == 2 ? D / 32 : c_first + D / 64;
        const uint32_t tA = tmem + C::kO + lane_off, tB = tA + D;  // the two results
#pragma unroll 1
        for (int c = c_first; c < c_last; ++c) {
          uint32_t w[32];
          if (nt == 2) {
            tc::ld32(tO + 32 * c, w);
            tc::wait_ld();
          } else {
            const float fa = wg ? f1 : f0, fb = wg ? f0 : f1;
            uint32_t y[32];
            tc::ld32(tA + 32 * c, w);
            tc::ld32(tB + 32 * c, y);
            tc::wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              w[k] = __float_as_uint(fmaf(__uint_as_float(y[k]), fb, __uint_as_float(w[k]) * fa));
          }
          if (any_bad) {  // the NaN that were taken out of V, to the rows that see them
            for (int k = 8 * b0; k < 8 * b1; ++k) {
              const int at = base + jt * kBN + k;
              if (!(bad[k >> 3] >> (k & 7) & 1) || !tree::sees_node(mask, at - e.P)) continue;
              const int blk = __ldg(table + (at >> sp.bs_shift));
              if (blk < 0 || int64_t(blk) >= p.num_blocks) continue;
              const unsigned char* s = p.v_group_scales + int64_t(blk) * p.ts_block + int64_t(kvh) * p.ts_head +
                                       (at & (p.block_size - 1)) * C::kGroups + 2 * c;
              const bool lo = (s[0] & 0x7f) == 0x7f, hi = (s[1] & 0x7f) == 0x7f;
#pragma unroll
              for (int u = 0; u < 32; ++u)
                if (u < 16 ? lo : hi) w[u] = 0x7fc00000u;
            }
          }
          if (!row_ok) continue;
          if (whole) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + trow * p.out_stride_t +
                                 int64_t(kvh * g + r_head) * p.out_stride_h + 32 * c;
            uint32_t o16[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const __nv_bfloat162 pr = __floats2bfloat162_rn(__uint_as_float(w[2 * k]) * inv,
                                                              __uint_as_float(w[2 * k + 1]) * inv);
              o16[k] = *reinterpret_cast<const uint32_t*>(&pr);
            }
            if (sp.out_vec) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint2*>(out + 4 * k) = make_uint2(o16[2 * k], o16[2 * k + 1]);
            } else {  // (rows at any address)
              uint16_t* o = reinterpret_cast<uint16_t*>(out);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                o[2 * k] = uint16_t(o16[k]);
                o[2 * k + 1] = uint16_t(o16[k] >> 16);
              }
            }
          } else {
            float4* o = reinterpret_cast<float4*>(sp.o + prow * D + 32 * c);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              o[k] = make_float4(__uint_as_float(w[4 * k]) * inv, __uint_as_float(w[4 * k + 1]) * inv,
                                 __uint_as_float(w[4 * k + 2]) * inv, __uint_as_float(w[4 * k + 3]) * inv);
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&st->bars[kOFree]);
    }
    if (!ok && lane == 0) {
      st->abort = 1;
      raise_device_error(p.err, kErrTimeout);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(tmem, kTmemCols);
}

}  // namespace tree_e2m1

namespace {

template <int D>
cudaError_t launch_tree_e2m1_tpl(const TreeParams& p, const TreeSplit& sp, cudaStream_t stream) {
  using C = tree_e2m1::Cfg<D>;
  static_assert(sizeof(tree_e2m1::State) <= C::kStateBytes, "state");
  static_assert(C::kSmem <= 227 * 1024, "shared memory");
  constexpr int kDevices = 64;
  auto kern = tree_e2m1::tree_e2m1_kernel<D>;
  static std::once_flag once[kDevices];
  static cudaError_t set[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    set[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem));
  });
  if (set[dev] != cudaSuccess) return set[dev];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sp.grid));
  cfg.blockDim = dim3(tree_e2m1::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p, sp);
  note_launch();
  if (e != cudaSuccess) return e;
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_tree_merge(p, sp, stream);
}

}  // namespace

bool tree_e2m1_supported(const TreeParams& p) {
  if (p.q_dtype != kBF16 || p.kv_dtype != kE2M1) return false;
  if (p.group > tree::kBM) return false;
  if ((p.cs_block | p.cs_head | p.ts_block | p.ts_head) >> 32 || p.num_blocks > 0x7fffffff) return false;  // (multiplied in 32 bits)
  return (reinterpret_cast<uintptr_t>(p.query) & 15) == 0 && (p.q_stride_t & 7) == 0 && (p.q_stride_h & 7) == 0;
}

cudaError_t launch_tree_e2m1(const TreeParams& p, TreeSplit sp, cudaStream_t stream) {
  sp.item_nodes = 2 * sp.tq;
  return p.head_dim == 128 ? launch_tree_e2m1_tpl<128>(p, sp, stream) : launch_tree_e2m1_tpl<64>(p, sp, stream);
}

}  // namespace pkv
