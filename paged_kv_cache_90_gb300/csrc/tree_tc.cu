// tree_tc.cu — attention of drafted token trees over the paged cache on the
// fifth-generation tensor cores (tcgen05 MMAs, accumulators in tensor memory).
//
// A KV head's K and V are read once for all the rows that use them: the group's g query
// heads times up to TQ = 128 / g (rounded down) drafted nodes make a row tile of 128 MMA
// rows (row r = node r / g, head r % g; the rest idle), and two row tiles share a pass
// over the keys.  With few rows the call is a stream of the cache and HBM bounds it; with
// 256 rows to a KV head the tensor work of a key tile (2 x 2 x 128 x 128 x D
// multiply-adds) takes as long as its bytes.
//
// Work split.  An item is (sequence, KV head, pair of row tiles); its work is its key
// tiles of 128 positions.  The items' tiles, laid end to end, are cut into equal
// contiguous ranges, one per SM, so one long context occupies the whole GPU and many
// short ones balance.  An item inside one range writes its output; one cut by a border
// leaves, per part, the rows' maximum, sum and unnormalised output in binary32, which a
// second small kernel folds in order (so the result never depends on timing).
//
// A step is one (key tile, row tile):
//   S = Q K^T        M 128, N 128, K = D: both from shared memory (128-byte swizzle), S in
//                    one of two tensor-memory buffers, by the step's parity
//   P = 2^(S c - m)  written back over S as bf16 pairs by a softmax warpgroup, a row per
//                    thread; masked positions become zero here
//   O += P V         M 128, N = D, K = 128 keys: P from tensor memory, V from shared memory
// The MMA thread issues S of step x + 1 before P V of step x, so the tensor cores work
// while a softmax runs.  Two softmax warpgroups: each owns one Q buffer and one O
// accumulator.  A pair's two row tiles go to the two of them; single row tiles alternate,
// so that one item's output is written while the next one's softmax runs.
//
// What it measured, 32 query heads to 8 KV heads of 128: 64 trees of 5 to 24 nodes over 160 to
// 2048 positions 62 us, 5.0 TB/s, bound by the copies in flight (a tile is 64 KB, the rings hold
// three and three) and by each block's start and end; 8 trees of 64 nodes over 32000 positions 240
// us, 1.10 PFLOP/s at the power limit: a tile's two steps take 3500 to 3900 clocks (a warpgroup's
// softmax 3000 beside the other's, and the MMA warp between them), an item's end and the next
// one's start 16000 more, so blocks with such a border end a tenth after the others.
//
// P is rounded to bf16 for the product (at most half a step, 2^-8 of a weight; the
// other operand is bf16); scores, maximum, sum and output stay in binary32.  The
// reference maximum moves only when a row's maximum grows by more than 2^8, as in the
// decode kernel.
//
// Warps: 0 streams K tiles, 2 V tiles (TMA), 3 the queries; 1 issues the
// MMAs; 4-7 and 8-11 are the softmax warpgroups; 12 cleans the V tiles at the ends of the
// contexts.  Every wait is bounded; when one runs
// out the block sets an error bit and a flag that makes every role stop, lets its copies
// and MMAs land and frees the tensor memory.
#include <algorithm>
#include <mutex>

#include "decode_mma_launch.cuh"
#include "tcgen05.cuh"
#include "tree_split.cuh"
#include "umma.cuh"

namespace pkv {
namespace tree_tc {

using namespace tree;

constexpr int kThreads = 416;
constexpr uint32_t kTmemCols = 512;

// Shared memory: slots of one operand tile (128 rows), for the queries, then a ring of K
// tiles and one of V tiles.  In-flight copies are what the HBM rate hangs on, so the second
// query slot goes to the K ring where no sequence has a second row tile.
template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;             // 64-column halves of an operand (128-byte rows)
  static constexpr uint32_t kHalfBytes = kBM * 128;  // 16 KB
  static constexpr uint32_t kOpBytes = kHalves * kHalfBytes;
  static constexpr int kSlots = D == 128 ? 7 : 13;
  __host__ __device__ static constexpr int k_ring(int q_slots) { return (kSlots - q_slots) / 2; }
  __host__ __device__ static constexpr int v_ring(int q_slots) { return kSlots - q_slots - k_ring(q_slots); }
  static constexpr uint32_t kState = kSlots * kOpBytes;
  static constexpr uint32_t kStateBytes = 2048;
  static constexpr size_t kSmem = kState + kStateBytes + 1024;  // (+ alignment)
  // tensor memory: S of even and odd steps (128 columns each), then O of the two slots
  static constexpr uint32_t kS = 0, kO = 2 * kBN;
};

// Barriers.  A wait names a phase by its parity, so its barrier may be at most one phase
// away: those that a softmax warpgroup waits for (S, and the products' completion) count its
// own slot's steps, two barriers a slot by the parity of the slot's step.  A warpgroup may wait
// for a step while the other one is several steps behind it, and for the last product of an
// item while the one before it is still held up by its V tile.
constexpr int kMaxRing = 6;
enum Bar { kQFull = 0, kQEmpty = 2, kKFull = 4, kKEmpty = kKFull + kMaxRing, kVFull = kKEmpty + kMaxRing,
           kVEmpty = kVFull + kMaxRing, kVRaw = kVEmpty + kMaxRing, kSFull = kVRaw + kMaxRing, kPFull = kSFull + 4,
           kODone = kPFull + 2, kOFree = kODone + 4, kDrain = kOFree + 2, kNumBars = kDrain + 1 };

constexpr int kBadItems = 8;  // items whose bad rows are kept: the cleaning warp is up to a ring of
                              // V tiles and one item ahead of a warpgroup that writes its output

// Small shared state behind the operands.
struct State {
  uint64_t bars[kNumBars + 1];
  volatile int abort;
  uint32_t tmem;
  Range range;
  longlong2 warp_sum[kThreads / 32];
  // drafted positions with an infinity or a NaN in V, 32 to a word from the first tile
  // that holds drafted nodes on (1024 nodes touch at most 9 tiles), per item (index mod
  // kBadItems)
  uint32_t bad_rows[kBadItems][36];
};
static_assert(sizeof(State) <= 2048, "state");

// Waits for barrier `bar`; by a whole warp: all its lanes see one answer.
__device__ __forceinline__ bool wait(State* st, int bar, uint32_t parity) {
  return tree::wait(&st->bars[bar], parity, &st->abort);
}
__device__ __forceinline__ bool wait_warp(State* st, int bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(st, bar, parity));
}

__device__ __forceinline__ bool ready(uint64_t* bar, uint32_t parity) {  // one answer for a warp
  return __all_sync(0xffffffffu, test_wait(bar, parity));
}

// Bits c0 .. c0 + 31 of a row's mask (its first word loaded beforehand): 1 for positions
// before the drafted nodes (c < 0), 0 behind them (c >= n).
__device__ __forceinline__ uint32_t mask_bits(const int64_t* mask, uint64_t word0, int c0, int n) {
  if (c0 >= n) return 0u;
  uint32_t past = 0u;
  int sh = 0;
  if (c0 < 0) {
    if (c0 <= -32) return 0xffffffffu;
    sh = -c0;
    past = (1u << sh) - 1u;
    c0 = 0;
  }
  const int w = c0 >> 6, o = c0 & 63;
  uint64_t b = (w == 0 ? word0 : uint64_t(__ldg(mask + w))) >> o;
  if (o > 32 && 64 * (w + 1) < n) b |= uint64_t(__ldg(mask + w + 1)) << (64 - o);
  const int valid = n - c0;
  uint32_t bits = uint32_t(b);
  if (valid < 32) bits &= (1u << valid) - 1u;
  return past | (bits << sh);
}

// The positions pos .. pos + 127 of a tile that a row sees, 64 to a word.
__device__ __forceinline__ void tile_bits(const tree::Extent& e, int pos, const int64_t* mask, uint64_t word0,
                                          uint64_t (&k)[2]) {
  auto ones = [](int n) -> uint64_t { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; };
  if (e.n <= 64) {
    // bits below sh are positions before the nodes, then come the nodes' bits
    const int sh = e.P - pos;
    const uint64_t m = word0 & ones(e.n);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int s = sh - 64 * w;
      k[w] = ones(s) | (s >= 64 || s <= -64 ? 0ull : s >= 0 ? m << s : m >> -s);
    }
  } else {
#pragma unroll 1
    for (int w = 0; w < 4; ++w) {
      const uint64_t b = mask_bits(mask, word0, pos + 32 * w - e.P, e.n);
      if (w & 1) k[w >> 1] |= b << 32; else k[w >> 1] = b;
    }
  }
}

// Largest of a row's 32 scores at tensor-memory column `ts`; with kCut those not kept
// become -infinity there.
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
  float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 32; ++i) t[i & 3] = fmaxf(t[i & 3], __uint_as_float(w[i]));
  return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

// Weights 2^(score * sl - mu) of a row's 32 scores at column `ts`, written as bf16 pairs to
// column `tp` (whose scores have been read); returns their sum.
__device__ __forceinline__ float weights(uint32_t ts, uint32_t tp, float sl, float mu) {
  uint32_t w[32], pk[16];
  tc::ld32(ts, w);
  tc::wait_ld();
  float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float a = fast_exp2(fmaf(__uint_as_float(w[2 * i]), sl, -mu));
    const float b = fast_exp2(fmaf(__uint_as_float(w[2 * i + 1]), sl, -mu));
    ps[i & 3] += a + b;
    const __nv_bfloat162 pr = __floats2bfloat162_rn(a, b);
    pk[i] = *reinterpret_cast<const uint32_t*>(&pr);
  }
  tc::st16(tp, pk);
  return (ps[0] + ps[1]) + (ps[2] + ps[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
               const __grid_constant__ CUtensorMap tmv, const __grid_constant__ TreeParams p, const TreeSplit sp) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  State* st = reinterpret_cast<State*>(smem + C::kState);
  // (the warp's number from one lane: the compiler then knows that it is the same in all, and what
  // follows from it, a role's loops and addresses, is computed once for the warp)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int g = p.group, TQ = sp.tq;
  const uint32_t sbase = smem_addr(smem);

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const bool warps4 = (i >= kPFull && i < kPFull + 2) || (i >= kOFree && i < kOFree + 2);
      mbar_init(&st->bars[i], warps4 ? 4 : 1);  // (one arrival per softmax warp)
    }
    st->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) tc::alloc(&st->tmem, kTmemCols);
  if (tid == 32) {  // the first copies find their maps near
    prefetch_map(&tmq);
    prefetch_map(&tmk);
    prefetch_map(&tmv);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing of the caller's is read before
  asm volatile("griddepcontrol.launch_dependents;");

  // (nq: query slots, two where some sequence of the batch has a second row tile)
  const int nq = find_range<kThreads>(p, sp, &st->range, st->warp_sum, sp.tq) ? 2 : 1;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = st->tmem;
  const Range* rg = &st->range;
  const int64_t from = rg->from;
  Walk it;
  it.start(p, sp, rg);
  const int kr = C::k_ring(nq), vr = C::v_ring(nq);
  const uint32_t sq = sbase, sk = sq + nq * C::kOpBytes, sv = sk + kr * C::kOpBytes;  // the slots

  if (warp == 0 || warp == 2) {
    // ---- K (warp 0) and V (warp 2) tiles: lane i issues copy i of a tile (one box of
    // `box` positions x one 64-column half), its table entry fetched a tile ahead ---------
    const bool isv = warp == 2;
    const int bs = p.block_size, box = min(bs, 16);
    const int eb = isv ? kVEmpty : kKEmpty, fb = isv ? kVFull : kKFull;
    const uint32_t region = isv ? sv : sk;
    const CUtensorMap* map = isv ? &tmv : &tmk;
    const int bx = lane / C::kHalves, half = lane % C::kHalves;
    const int ring = isv ? vr : kr;
    int kt = 0, slot = 0;    // tile, its slot
    uint32_t phase = 0;      // and the parity of the slot's use
    // tile j of `it` is looked up (its entry loaded) one tile before its copy is issued, over
    // the borders of items too
    int j = it.valid() ? it.j0 : 0, pos = 0, kvh = 0, nbox = 0, e = 0, bar = fb;
    uint32_t raw = 0;        // the slots whose last copy went to the cleaning warp,
    uint32_t raw_phase = 0;  // and the parities of their uses by it
    bool have = false;
    while (true) {
      const int pos0 = pos, kvh0 = kvh, nbox0 = nbox, e0 = e, bar0 = bar;
      const bool copy = have;
      have = it.valid();
      if (have) {
        pos = it.q.base + j * kBN;
        kvh = it.kvh;
        nbox = max(0, min(kBN, it.q.e.L - pos) + box - 1) / box;  // (the tile's boxes end at L)
        bar = isv && it.cut(j) ? kVRaw : fb;
        e = 0;
        if (bx < nbox) e = __ldg(p.block_tables + int64_t(it.s) * p.bt_stride + ((pos + bx * box) >> sp.bs_shift));
        if (++j == it.j1) {
          it.next(p, sp, rg);
          j = it.j0;
        }
      }
      if (copy) {
        bool ok = true;
        if (lane == 0 && kt >= ring) ok = wait(st, eb + slot, phase ^ 1u);
        if (!__shfl_sync(0xffffffffu, int(ok), 0)) break;
        if (lane == 0) mbar_arrive_expect_tx(&st->bars[bar0 + slot], uint32_t(nbox0 * box) * 128u * C::kHalves);
        __syncwarp();
        raw = bar0 == kVRaw ? raw | 1u << slot : raw & ~(1u << slot);
        if (bar0 == kVRaw) raw_phase ^= 1u << slot;
        if (bx < nbox0) {
          int blk = e0;
          if (blk < 0 || int64_t(blk) >= p.num_blocks) {
            raise_device_error(p.err, kErrTableEntry);
            blk = 0;
          }
          tma_4d(region + slot * C::kOpBytes + half * C::kHalfBytes + uint32_t(bx * box * 128), map, 64 * half,
                 (pos0 + bx * box) & (bs - 1), kvh0, blk, &st->bars[bar0 + slot]);
        }
        ++kt;

        if (++slot == ring) {
          slot = 0;
          phase ^= 1u;
        }
      } else if (!have) {
        break;
      }
    }
    // the copies in flight land before the block may exit
    if (lane == 0)
      for (int k = max(0, kt - ring); k < kt; ++k) {
        const int s = k % ring;
        if (raw >> s & 1u) (void)mbar_wait_bounded(&st->bars[kVRaw + s], (raw_phase >> s & 1u) ^ 1u);
        else (void)mbar_wait_bounded(&st->bars[fb + s], uint32_t(k / ring) & 1u);
      }
  } else if (warp == 3) {
    // ---- queries: the row tiles of each item, alternating between the two slots; and what
    // the fold needs of an item that goes on in the next block's range --------------------
    if (lane == 0) {
      int oc = 0, uses0 = 0, uses1 = 0;  // of the slots
      bool ok = true;
      int64_t at = from;
      TreeSplit::Tail tail = {0, 0, 0, 0};
      for (; ok && it.valid(); it.next(p, sp, rg)) {
        for (int qt = 0; ok && qt < it.nt; ++qt, ++oc) {
          const int slot = oc & (nq - 1), n = slot ? uses1 : uses0;
          if (n > 0) ok = wait(st, kQEmpty + slot, uint32_t(n - 1) & 1u);
          if (!ok) break;
          if (slot) ++uses1; else ++uses0;
          mbar_arrive_expect_tx(&st->bars[kQFull + slot], uint32_t(g * sp.q_nodes) * 128u * C::kHalves);
          for (int h = 0; h < C::kHalves; ++h)
            tma_3d(sq + slot * C::kOpBytes + h * C::kHalfBytes, &tmq, 64 * h, it.kvh * g,
                   it.q.e.q0 + (2 * it.pair + qt) * TQ, &st->bars[kQFull + slot]);
        }
        if (it.begins() && !it.ends()) {
          const int node0 = 2 * it.pair * TQ;
          tail.row0 = it.q.e.q0 + node0;
          tail.nodes = min(2 * TQ, it.q.e.n - node0);
          tail.kvh = it.kvh;
          tail.last = int((at - it.u0 + it.q.tiles + rg->cost - 1) / rg->share);
        }
        at += it.u1 - it.u0;
      }
      sp.tails[blockIdx.x] = tail;
      if (uses0) (void)mbar_wait_bounded(&st->bars[kQFull], uint32_t(uses0 - 1) & 1u);
      if (uses1) (void)mbar_wait_bounded(&st->bars[kQFull + 1], uint32_t(uses1 - 1) & 1u);
    }
  } else if (warp == 1) {
    // ---- MMAs (a warp, see umma.cuh): S runs up to two steps ahead of P V; whichever can go next
    // goes, so that neither a late key tile nor a late softmax holds up the other ----------
    {
      constexpr uint32_t idS = tc::idesc_bf16(kBM, kBN, 0, 0);
      constexpr uint32_t idO = tc::idesc_bf16(kBM, D, 0, 1);
      constexpr uint64_t kOp = C::kOpBytes >> 4;  // (descriptors hold addresses / 16)
      const uint64_t qdesc = tc::desc_sw128(sq, 16, 1024), kdesc = tc::desc_sw128(sk, 16, 1024);
      const uint64_t vdesc = tc::desc_sw128(sv, C::kHalfBytes, 1024);
      // a step between its S and its P V: what the P V needs to know
      struct Pending {
        bool slot, odd, x, x_phase, first, last_tile, wait_o, o_phase, v_phase;
        uint8_t v;  // V slot
      };
      Pending pend[2];  // [step & 1] (constant indices below: registers)
      int xs = 0, xp = 0;   // next step of either kind
      int j = it.j0, qt = 0, oc = 0, uses0 = 0, uses1 = 0, steps0 = 0, steps1 = 0;
      int ks = 0, vs = 0;             // K and V slot of the tile
      uint32_t kp = 0;                // and the parities of the slots' uses
      bool vp = false;
      uint32_t idle = 0;
      bool ok = true;
      while (it.valid() || xp < xs) {
        bool went = false;
        if (it.valid() && xs <= xp + 1 && ready(&st->bars[kKFull + ks], kp)) {
          const int slot = (oc + qt) & 1, u = slot ? uses1 : uses0, n = slot ? steps1 : steps0;
          const int qs = slot & (nq - 1);  // (with one query slot its uses are those of both O slots)
          if (j > it.j0 || ready(&st->bars[kQFull + qs], uint32_t(nq == 2 ? u : uses0 + uses1) & 1u)) {
            tc::fence_after();
            const uint64_t qd = qdesc + qs * kOp, kd = kdesc + ks * kOp;
            const uint32_t ts = tmem + C::kS + (xs & 1) * kBN;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              constexpr uint64_t kHalf = C::kHalfBytes >> 4;
              const uint64_t off = (kk >> 2) * kHalf + (kk & 3) * 2;
              umma::mma_ss(ts, qd + off, kd + off, idS, kk > 0 ? 1u : 0u);
            }
            umma::commit(&st->bars[kSFull + 2 * slot + (n & 1)]);
            const bool last_row_tile = qt == it.nt - 1;
            if (last_row_tile) umma::commit(&st->bars[kKEmpty + ks]);
            if (j == it.j1 - 1) umma::commit(&st->bars[kQEmpty + qs]);
            const Pending pd = {slot != 0, (n & 1) != 0, (xs & 1) != 0, ((xs >> 1) & 1) != 0, j == it.j0, last_row_tile,
                                j == it.j0 && u > 0, ((u - 1) & 1) != 0, vp, uint8_t(vs)};
            if (xs & 1) pend[1] = pd; else pend[0] = pd;
            ++xs;
            if (slot) ++steps1; else ++steps0;
            if (!last_row_tile) {
              ++qt;
            } else {
              qt = 0;
              if (++ks == kr) {
                ks = 0;
                kp ^= 1u;
              }
              if (++vs == vr) {
                vs = 0;
                vp = !vp;
              }
              if (++j == it.j1) {
                if (it.nt == 2 || (oc & 1) == 0) ++uses0;
                if (it.nt == 2 || (oc & 1) == 1) ++uses1;
                oc += it.nt;
                it.next(p, sp, rg);
                j = it.j0;
              }
            }
            went = true;
          }
        }
        if (xp < xs) {
          const Pending pd = (xp & 1) ? pend[1] : pend[0];
          if (ready(&st->bars[kPFull + pd.x], pd.x_phase) && ready(&st->bars[kVFull + pd.v], pd.v_phase) &&
              (!pd.wait_o || ready(&st->bars[kOFree + pd.slot], pd.o_phase))) {
            tc::fence_after();
            const uint64_t vd = vdesc + pd.v * kOp;
            const uint32_t ts = tmem + C::kS + pd.x * kBN, to = tmem + C::kO + pd.slot * D;
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk)
              umma::mma_ts(to, ts + 8 * kk, vd + kk * (16 * 128 >> 4), idO, (!pd.first || kk > 0) ? 1u : 0u);
            umma::commit(&st->bars[kODone + 2 * pd.slot + pd.odd]);
            if (pd.last_tile) umma::commit(&st->bars[kVEmpty + pd.v]);
            ++xp;
            went = true;
          }
        }
        if (went) {
          idle = 0;
        } else {
          __nanosleep(20);  // (a spinning thread takes issue slots from the softmax beside it)
          if ((++idle & 255u) == 0 && (st->abort || idle > kWaitPolls)) {
            ok = false;
            break;
          }
        }
      }
      // every MMA issued has completed before the tensor memory is freed
      umma::commit(&st->bars[kDrain]);
      (void)mbar_wait_bounded(&st->bars[kDrain], 0);
      if (!ok) {
        st->abort = 1;
        if (lane == 0) raise_device_error(p.err, kErrTimeout);
      }
    }
  } else if (warp == 12) {
    // ---- tiles with positions that are hidden from some row: V rows past the sequence's end
    // are zeroed in shared memory (they may hold anything), and infinities and NaN of drafted
    // nodes taken out of it (0 x infinity would reach the rows that do not see the node; those
    // that do get them back with the output) -------------------------------------------------
    int slot = 0, item = 0;
    uint32_t phase = 0;  // parities of the slots' uses by this warp
    bool ok = true;
    for (; ok && it.valid(); it.next(p, sp, rg), ++item) {
      const tree::Extent& e = it.q.e;
      const int jt = (e.P - it.q.base) / kBN;  // first tile with drafted nodes
      for (int j = it.j0; j < it.j1; ++j, slot = slot + 1 == vr ? 0 : slot + 1) {
        if (!it.cut(j)) continue;
        // (such a tile's copies complete on a barrier of its own; the MMA thread sees the
        // tile when this warp passes it on)
        const int pos = it.q.base + j * kBN;
        if (!(ok = wait_warp(st, kVRaw + slot, phase >> slot & 1u))) break;
        phase ^= 1u << slot;
        unsigned char* vt = smem + (sv - sbase) + slot * C::kOpBytes;
        constexpr int kCells = 8 * C::kHalves;  // 16-byte cells of a row
        auto cell = [&](int i) {  // (row i / kCells)
          return reinterpret_cast<uint4*>(vt + ((i >> 3) % C::kHalves) * C::kHalfBytes + (i / kCells) * 128 + (i & 7) * 16);
        };
        const int hi = max(0, min(kBN, e.L - pos));
        for (int i = hi * kCells + lane; i < kBN * kCells; i += 32) *cell(i) = make_uint4(0u, 0u, 0u, 0u);
        for (int q = 0; q < 4; ++q) {  // the drafted nodes, 32 positions to a word
          const int end = min(hi, 32 * q + 32) * kCells;
          uint32_t bad = 0u;
          // (four loads together: one after the other they take longer than the tile's products)
#pragma unroll 1
          for (int i0 = max(e.P - pos, 32 * q) * kCells + lane; i0 < end; i0 += 128) {
            uint4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = i0 + 32 * u < end ? *cell(i0 + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
              bool any = false;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((w[k] & 0x7f80u) == 0x7f80u) { w[k] &= 0xffff0000u; any = true; }
                if ((w[k] & 0x7f800000u) == 0x7f800000u) { w[k] &= 0xffffu; any = true; }
              }
              if (any) {
                *cell(i0 + 32 * u) = make_uint4(w[0], w[1], w[2], w[3]);
                bad |= 1u << (((i0 + 32 * u) / kCells) & 31);
              }
            }
          }
          bad = __reduce_or_sync(0xffffffffu, bad);
          if (lane == 0) st->bad_rows[item % kBadItems][4 * (j - jt) + q] = bad;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->bars[kVFull + slot]);
      }
    }
    if (!ok && lane == 0) {
      st->abort = 1;
      raise_device_error(p.err, kErrTimeout);
    }
  } else if (warp >= 4) {
    // ---- softmax warpgroup `wg` (slot wg): row r of its row tiles, r = tensor-memory lane --
    const int wg = (warp >> 2) - 1, q = warp & 3;
    const int r = 32 * q + lane, r_node = r / g, r_head = r - r_node * g;
    const uint32_t lane_off = uint32_t(32 * q) << 16;
    const uint32_t tO = tmem + C::kO + wg * D + lane_off;
    const float sl = p.qk_scale_log2;
    int x0 = 0, oc = 0, item = 0, steps = 0;  // `steps`: of this slot so far
    bool ok = true;
    for (; ok && it.valid(); x0 += (it.j1 - it.j0) * it.nt, oc += it.nt, ++item, it.next(p, sp, rg)) {
      const int qt = (oc & 1) == wg ? 0 : 1;
      if (qt >= it.nt) continue;
      const tree::Extent& e = it.q.e;
      const int node = (2 * it.pair + qt) * TQ + r_node;
      const bool row_ok = r < TQ * g && node < e.n;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      const int64_t trow = e.q0 + node;
      const int64_t* mask = p.tree_mask + (row_ok ? trow : int64_t(e.q0)) * p.mask_stride;  // (idle rows: any)
      const uint64_t word0 = uint64_t(__ldg(mask));
      const uint32_t* bad_rows = st->bad_rows[item % kBadItems];
      const int jt = (e.P - it.q.base) / kBN;  // first tile with drafted nodes
      float m_ref = -INFINITY, l_run = 0.f;
      for (int j = it.j0; j < it.j1; ++j, ++steps) {
        const int x = x0 + (j - it.j0) * it.nt + qt;
        const int pos = it.q.base + j * kBN;
        const uint32_t tS = tmem + C::kS + (x & 1) * kBN + lane_off;
        if (!(ok = wait_warp(st, kSFull + 2 * wg + (steps & 1), uint32_t(steps >> 1) & 1u))) break;
        tc::fence_after();
        const bool cut = it.cut(j);
        if (warp_ok) {
          float mx = -INFINITY;
          if (cut) {
            uint64_t k[2];
            tile_bits(e, pos, mask, word0, k);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              mx = fmaxf(mx, row_max<true>(tS + 32 * c, uint32_t(k[0])));
              k[0] = k[0] >> 32 | k[1] << 32;
              k[1] >>= 32;
            }
            tc::wait_st();
          } else {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) mx = fmaxf(mx, row_max<false>(tS + 32 * c, 0u));
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
              for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
              tc::st32(tO + 32 * c, w);
            }
            tc::wait_st();
            l_run *= alpha;
          }
          if (move) m_ref = mx;
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          float sum = 0.f;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) sum += weights(tS + 32 * c, tS + 16 * c, sl, mu);
          l_run += sum;
          tc::wait_st();
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->bars[kPFull + (x & 1)]);
      }
      if (!ok) break;
      // ---- the part's output ---------------------------------------------------------------
      if (!(ok = wait_warp(st, kODone + 2 * wg + ((steps - 1) & 1), uint32_t((steps - 1) >> 1) & 1u))) break;
      tc::fence_after();
      if (warp_ok) {
        const bool whole = it.begins() && it.ends();
        const float inv = whole ? (l_run != 0.f ? 1.f / l_run : 0.f) : 1.f;
        const int64_t prow = int64_t(2 * blockIdx.x + (it.begins() ? 1 : 0)) * sp.rows + qt * kBM + r;
        if (row_ok && !whole) sp.ml[prow] = make_float2(m_ref, l_run);
        // (the words of this part's tiles; the others are not this item's)
        const int bw0 = 4 * (max(it.j0, jt) - jt), bw1 = 4 * (it.j1 - jt);
        bool any_bad = false;
        if (row_ok)
          for (int w = bw0; w < bw1; ++w) any_bad |= bad_rows[w] != 0u;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[32];
          tc::ld32(tO + 32 * c, w);
          tc::wait_ld();
          if (any_bad) {
            // add what was taken out of V to the rows that see it
            for (int k = 32 * bw0; k < 32 * bw1; ++k) {
              const int at = it.q.base + jt * kBN + k;
              if (!(bad_rows[k >> 5] >> (k & 31) & 1u) || !tree::sees_node(mask, at - e.P)) continue;
              const int blk = __ldg(p.block_tables + int64_t(it.s) * p.bt_stride + (at >> sp.bs_shift));
              if (blk < 0 || int64_t(blk) >= p.num_blocks) continue;
              const uint16_t* v = static_cast<const uint16_t*>(p.value_cache) + int64_t(blk) * p.cs_block +
                                  int64_t(it.kvh) * p.cs_head + int64_t(at & (p.block_size - 1)) * D + 32 * c;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((v[i] & 0x7f80u) == 0x7f80u) w[i] = __float_as_uint(__uint_as_float(w[i]) + bf16_lo_to_f32(v[i]));
            }
          }
          if (!row_ok) continue;
          if (whole) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + trow * p.out_stride_t +
                                 int64_t(it.kvh * g + r_head) * p.out_stride_h + 32 * c;
            uint32_t o16[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const __nv_bfloat162 pr = __floats2bfloat162_rn(__uint_as_float(w[2 * i]) * inv,
                                                              __uint_as_float(w[2 * i + 1]) * inv);
              o16[i] = *reinterpret_cast<const uint32_t*>(&pr);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(out + 8 * i) =
                  make_uint4(o16[4 * i], o16[4 * i + 1], o16[4 * i + 2], o16[4 * i + 3]);
          } else {
            uint4* o = reinterpret_cast<uint4*>(sp.o + prow * D + 32 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&st->bars[kOFree + wg]);
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

}  // namespace tree_tc

namespace {

// 3-D map over the queries [T, Hq, D]: box = 64 columns x the group's heads x `nodes` rows,
// 128-byte swizzle.
cudaError_t make_tree_query_map(CUtensorMap* map, const TreeParams& p, int nodes) {
  auto fn = tensor_map_encoder();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {cuuint64_t(p.head_dim), cuuint64_t(p.num_heads), cuuint64_t(p.num_tokens)};
  // (the stride of a dimension of one may be anything)
  const int64_t sh = p.num_heads > 1 ? p.q_stride_h : p.head_dim;
  const int64_t st = p.num_tokens > 1 ? p.q_stride_t : sh * p.num_heads;
  const cuuint64_t strides[2] = {cuuint64_t(sh) * 2, cuuint64_t(st) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(p.group), cuuint32_t(nodes)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.query), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_tree_tc_tpl(const TreeParams& p, TreeSplit sp, cudaStream_t stream) {
  using C = tree_tc::Cfg<D>;
  CUtensorMap mq, mk, mv;
  sp.item_nodes = 2 * sp.tq;
  // the tile's rows that can hold nodes: no more than the batch has
  sp.q_nodes = int(std::min<int64_t>(tree::kBM / p.group, p.num_tokens));
  cudaError_t e = make_tree_query_map(&mq, p, sp.q_nodes);
  if (e != cudaSuccess) return e;
  DecodeParams dp{};  // (what the cache maps are made from)
  dp.kv_dtype = p.kv_dtype;
  dp.head_dim = p.head_dim;
  dp.block_size = p.block_size;
  dp.num_kv_heads = p.num_kv_heads;
  dp.num_blocks = p.num_blocks;
  dp.cs_head = p.num_kv_heads > 1 ? p.cs_head : int64_t(p.block_size) * p.head_dim;
  dp.cs_block = p.num_blocks > 1 ? p.cs_block : dp.cs_head * p.num_kv_heads;
  const int box = std::min(p.block_size, 16);
  if ((e = cached_cache_map(&mk, p.key_cache, dp, box)) != cudaSuccess) return e;
  if ((e = cached_cache_map(&mv, p.value_cache, dp, box)) != cudaSuccess) return e;
  auto kern = tree_tc::tree_tc_kernel<D>;
  static std::once_flag once[kMapCacheDevices];
  static cudaError_t set[kMapCacheDevices];
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= kMapCacheDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    set[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kSmem));
  });
  if (set[dev] != cudaSuccess) return set[dev];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sp.grid));
  cfg.blockDim = dim3(tree_tc::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, p, sp);
  note_launch();
  if (e != cudaSuccess) return e;
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_tree_merge(p, sp, stream);
}

}  // namespace

// (a bf16 cache comes with the tree call: there is always a mask and never a window)
bool tree_tc_supported(const TreeParams& p) {
  if (p.q_dtype != kBF16 || p.kv_dtype != kBF16) return false;
  if (!(p.block_size == 8 || p.block_size == 16 || p.block_size == 32)) return false;
  if (p.group > tree::kBM) return false;
  if (!(p.qk_scale_log2 > 0.f)) return false;  // (the maximum is taken before the scale)
  // tensor maps take no stride of 0 (expanded views)
  if ((p.num_heads > 1 && p.q_stride_h == 0) || (p.num_tokens > 1 && p.q_stride_t == 0)) return false;
  if ((p.num_kv_heads > 1 && p.cs_head == 0) || (p.num_blocks > 1 && p.cs_block == 0)) return false;
  if ((reinterpret_cast<uintptr_t>(p.query) & 15) || (p.q_stride_t & 7) || (p.q_stride_h & 7)) return false;
  if ((reinterpret_cast<uintptr_t>(p.out) & 15) || (p.out_stride_t & 7) || (p.out_stride_h & 7)) return false;
  return tensor_map_encoder() != nullptr;
}

cudaError_t launch_tree_merge(const TreeParams& p, const TreeSplit& sp, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sp.grid), unsigned((sp.rows + tree::kMergeRows - 1) / tree::kMergeRows));
  cfg.blockDim = dim3(tree::kMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = p.head_dim == 128 ? cudaLaunchKernelEx(&cfg, tree::tree_merge_kernel<128>, p, sp)
                                          : cudaLaunchKernelEx(&cfg, tree::tree_merge_kernel<64>, p, sp);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// (an entry that is out of range is read as block 0: the host refuses a cache without blocks)
bool tree_tensor_supported(const TreeParams& p) { return tree_tc_supported(p) || tree_i8_supported(p); }

// Rows of a part's slot: the batch's, or at most one row tile of 128 (int8 cache) or two.
int tree_part_rows(int64_t num_tokens, int group, bool decode, bool one_tile) {
  const int tq = tree::kBM / group;
  if (decode) return group;
  return num_tokens <= tq ? int(num_tokens) * group : (one_tile ? 1 : 2) * tree::kBM;
}

size_t tree_workspace(int grid, int rows, int head_dim) {
  return TreeSplit::kHeader + size_t(grid) * 2 * rows * (size_t(head_dim) + 2) * 4;
}

cudaError_t launch_tree_tensor(const TreeParams& p, int grid, int rows, void* ws, cudaStream_t stream) {
  TreeSplit sp{};
  sp.grid = grid;
  sp.rows = rows;
  sp.tq = tree::kBM / p.group;
  sp.bs_shift = 0;
  while ((1 << sp.bs_shift) < p.block_size) ++sp.bs_shift;
  sp.out_vec = (reinterpret_cast<uintptr_t>(p.out) & 7) == 0 && (p.out_stride_t & 3) == 0 && (p.out_stride_h & 3) == 0;
  unsigned char* w = static_cast<unsigned char*>(ws);
  // (the first words of the workspace are the decode kernel's counters, zero between calls)
  sp.tails = reinterpret_cast<TreeSplit::Tail*>(w + kWorkspaceHeader);
  sp.o = reinterpret_cast<float*>(w + TreeSplit::kHeader);
  sp.ml = reinterpret_cast<float2*>(sp.o + size_t(grid) * 2 * rows * p.head_dim);
  if (decode_i8_supported(p)) return launch_decode_i8(p, sp, stream);
  if (p.kv_dtype == kI8) return launch_tree_i8(p, sp, stream);
  return p.head_dim == 128 ? launch_tree_tc_tpl<128>(p, sp, stream) : launch_tree_tc_tpl<64>(p, sp, stream);
}

}  // namespace pkv
