// tree_i8.cu — attention of drafted trees (and decode of more than 16 heads a KV head) over a
// token-scaled int8 cache on the fifth-generation tensor cores.
//
// A cached token is head_dim codes and one scale.  With the MMA's 128 rows on the tokens of a
// key tile and its columns on the query rows (drafted nodes x the group's heads, up to 128),
// a token's two scales belong to one thread, the work of a softmax grows with the rows that
// there are, and few rows cost little:
//   S^T = K Q^T         M = 128 tokens, N = rows, K = D: K codes widened to f16 and Q (f16) in
//                       shared memory, S^T in tensor memory, lane = token
//   P^T = 2^(S ks c - m) vs   by one thread per token, written to shared memory as f16 (m: see below)
//   O^T += V^T P^T      M = D, N = rows, K = 128 tokens: V codes widened to f16, O^T in
//                       tensor memory, lane = column of the head
// The rows are shared by two softmax warpgroups (one, if there are at most 16); every key tile is
// widened once for all of them, and one MMA has all their rows.
//
// The codes are whole numbers, so f16 holds them exactly; a query row is scaled by a power of
// two that brings its largest element to 2^14, so its bf16 values are exact down to 2^-29 of
// that.  A weight times its value scale is rounded to f16, relative to a row's reference m: the
// largest of score + log2 of the value scale (i8::scale_exponent) among the tokens that the row
// sees, so neither a token of little weight nor a hidden one takes bits from the rest, whatever
// its scale.  Half a step, 2^-11, down to 2^-20 of the row's largest product, 2^-31 of that below.
// Sum, scores and output stay in binary32.  A reference moves when a row's largest exceeds it by
// 2^8: whether any thread of the warpgroup saw that is one barrier per tile (a thread adds its
// token's exponent once, to the largest of its rows), and only then are the maxima looked for.
//
// A tile is 2 x 128 x (D + 4) bytes from HBM, and 2 x 128 x D codes to widen: about 27 warp
// instructions for 512 codes (an exclusive-or, two byte permutes and two subtractions for four
// codes), one warpgroup's whole work.  The chain of a tile bounds it, not a unit: of 64 rows a
// warp's weights take 2600 clocks, what is between two tiles' weights (a signal, a wait, the
// scales) another 1500, with two S^T buffers so that the score MMAs are not part of it.  32 trees
// of 8 to 32 nodes, 4 x 8 heads of 128, over 1000 to 8192 positions: 169 us, 282 TFLOP/s.  It was
// 249 us with a pass over the scores before the weights, with products of each half of the rows
// (their A operand was read twice), and with the queries converted by one warp (33000 clocks
// between two items), and 195 with each thread working out its output rows' addresses.
//
// Warps: 0 streams K codes and the scales, 3 V codes (bulk copies of one (block, head) run each);
// 1 issues the score MMAs, 2 the products'; 4-7 and 8-11 are the softmax warpgroups, which also
// bring the queries in; 12-15 widen K, 16-19 V.  Every wait is bounded; when one runs out the
// block sets an error bit and a flag, every role runs through its loops without waiting, lets its
// copies and MMAs land and frees the tensor memory.

#include <algorithm>
#include <mutex>

#include "i8_codes.cuh"
#include "tcgen05.cuh"
#include "tree_split.cuh"
#include "umma.cuh"

namespace pkv {
namespace tree_i8 {

using namespace tree;

constexpr int kThreads = 640;
// registers of a thread, by warpgroup: launched with 96 each (5 x 96 = 480), then split anew
// into control, two softmax and two widening warpgroups (64 + 2 x 152 + 2 x 56 = 480)
constexpr int kRegsControl = 64, kRegsSoftmax = 152, kRegsWiden = 56;
static_assert(kRegsControl + 2 * kRegsSoftmax + 2 * kRegsWiden <= 5 * 96, "registers");
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxSlots = 16;  // of the ring of code tiles
constexpr int kFewRows = 16;   // rows that one warpgroup takes alone
constexpr int kHalfRows = 64;  // rows of a warpgroup at most

template <int D>
struct Cfg {
  // Widened operands go in units of 16 KB, two buffers for K and two for V, so that one is
  // filled while the MMAs read the other.  At D = 128 a tile is two units: of K, 64 columns of
  // the 128 tokens (half of the MMA's K); of V, 64 tokens with both halves of their columns.
  // At D = 64 it is one.
  static constexpr int kUnits = D / 64;
  static constexpr uint32_t kUnitBytes = kBN * 128;
  static constexpr int kVTokens = kBN / kUnits;             // of a unit of V
  static constexpr uint32_t kVHalf = kVTokens * 128;        // pitch of its 64-column halves
  static constexpr uint32_t kCodeBytes = kBN * D;
  static constexpr uint32_t kPBytes = kBN * 128;
  // from the 1024-aligned base: K units | V units | Q | P (two times 64 rows) | ring of code tiles |
  // state
  static constexpr uint32_t kK = 0, kV = 2 * kUnitBytes, kQ = 4 * kUnitBytes, kQUnit = kBN * 128;
  static constexpr uint32_t kP = kQ + kUnits * kQUnit, kCodes = kP + 2 * kPBytes;
  static constexpr uint32_t kState = 211 * 1024;
  static constexpr uint32_t kStateBytes = 15 * 1024;
  // slots of the ring, K and V in turn: an even number, so that a loader and the widening warps it
  // feeds have slots of their own and see every phase of their barriers
  static constexpr int kSlots = int((kState - kCodes) / kCodeBytes) & ~1;
  static constexpr size_t kSmem = kState + kStateBytes + 1024;  // (+ alignment)
  // tensor memory: S^T [2], then O^T [2], 128 columns each
  static constexpr uint32_t kS = 0, kO = 256;
};

constexpr int kScaleSlots = 8;  // tiles whose scales are in shared memory

enum Bar { kQFull = 0, kCodeFull, kCodeEmpty = kCodeFull + kMaxSlots, kKFull = kCodeEmpty + kMaxSlots,
           kKEmpty = kKFull + 2, kVFull = kKEmpty + 2, kVEmpty = kVFull + 2, kScaleFull = kVEmpty + 2,
           kScaleEmpty = kScaleFull + kScaleSlots, kSFull = kScaleEmpty + kScaleSlots, kPFull = kSFull + 2,
           kODone = kPFull + 2, kOFree = kODone + 2, kDrain = kOFree + 2, kNumBars = kDrain + 2 };

// What a warpgroup keeps of its rows.
struct alignas(16) Rows {
  float m[kHalfRows];      // reference (base 2), -infinity before the first score
  float lift[kHalfRows];   // kTopWeight - m; where m is infinite kNoLift, with which every score moves it
  float old[kHalfRows];    // the last move's lift before it
  float alpha[kHalfRows];  // the last move's factor on the sum and the output
  float part[4][16];       // of a reduction over the tokens: each warp's
};

constexpr float kNoLift = 3.402823466e38f;
constexpr float kTop = 100.f;  // a weight's exponent at most, so that it can be taken back

struct State {
  uint64_t bars[kNumBars + 1];
  volatile int abort;
  uint32_t tmem;
  Range range;
  longlong2 warp_sum[kThreads / 32];
  alignas(16) float qf[2][2][kHalfRows];  // a row's score factor, per item (index mod 2)
  Rows rows[2];
  alignas(16) float scales[kScaleSlots][2][kBN];  // of K and of V
};

// A wait that runs out tells the others and is not one for the loops to stop at: a role
// whose waits fail runs through its loops, so that barriers among warps always meet.
__device__ __forceinline__ bool wait(State* st, int bar, uint32_t parity) {
  return tree::wait(&st->bars[bar], parity, &st->abort);
}

// By a whole warp: one answer.
__device__ __forceinline__ bool wait_warp(State* st, int bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(st, bar, parity));
}

// The rows of a Walk's item: rows, row halves' size (a multiple of 16) and halves in use.
struct ItemRows {
  int rows, half, groups;
  __device__ __forceinline__ ItemRows(const TreeParams& p, const TreeSplit& sp, const Walk& it) {
    rows = min(sp.item_nodes, it.q.e.n - it.pair * sp.item_nodes) * p.group;
    groups = rows <= kFewRows ? 1 : 2;
    half = groups == 1 ? kFewRows : ((rows + 31) >> 5) << 4;
  }
};

// f16 x f16 -> f32, M x N, A and B K-major (0) or MN-major (1)
__device__ __forceinline__ uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// 512 chunks of 16 codes -> one unit of an operand (128-byte rows of 64 columns, swizzled), four
// to each thread of a widening warpgroup: the first from `src` to bytes `lo` and `hi` of shared
// memory, the others a, b and a + b further (`da`, `db`: multiples of 8 rows, so the swizzle
// stays).
__device__ __forceinline__ void widen_unit(const unsigned char* src, uint32_t a, uint32_t b, unsigned char* lo,
                                           unsigned char* hi, uint32_t da, uint32_t db) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t so = (i & 1 ? a : 0) + (i & 2 ? b : 0), to = (i & 1 ? da : 0) + (i & 2 ? db : 0);
    const uint4 c = *reinterpret_cast<const uint4*>(src + so);
    const uint2 x = i8::widen4(c.x), y = i8::widen4(c.y), z = i8::widen4(c.z), w = i8::widen4(c.w);
    *reinterpret_cast<uint4*>(lo + to) = make_uint4(x.x, x.y, y.x, y.y);
    *reinterpret_cast<uint4*>(hi + to) = make_uint4(z.x, z.y, w.x, w.y);
  }
}

// Two binary32 numbers in one register pair, and the operations that take both at once.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Asynchronous copies of one float and of four, or of zeros.
__device__ __forceinline__ void copy4(float* dst, const float* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
}

__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

template <int N>
__device__ __forceinline__ void less_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ bool group_any(int id, bool x) {  // over a warpgroup, with a barrier
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r) : "r"(uint32_t(x)), "r"(id) : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
  tc::wait_ld();
}

__device__ __forceinline__ void lds16(const float* s, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(s)[i];
    f[4 * i] = v.x;
    f[4 * i + 1] = v.y;
    f[4 * i + 2] = v.z;
    f[4 * i + 3] = v.w;
  }
}

// A softmax warpgroup's thread: token 32 warp + lane of the tile.
struct Token {
  int id;          // the warpgroup's barrier
  int warp, lane;  // of the warpgroup
  float ks, vs;    // the token's scales
  float ex;        // the value scale's exponent
  bool valid;      // the token is a position of the row's range
  bool cut;        // a tile where some row may not see some token: `keep` has this one's rows
  uint64_t keep;
};

// The sums of a thread's rows, 16 to an array so that loops over the rows need no unrolling
// (unrolled code misses the instruction cache at every tile): a register array takes constant
// indices only.
struct Sums {
  uint64_t a[4][8];
  template <typename F>
  __device__ __forceinline__ void chunk(int c, F f) {
    if (c == 0) f(a[0]);
    else if (c == 1) f(a[1]);
    else if (c == 2) f(a[2]);
    else f(a[3]);
  }
};

__device__ __forceinline__ float min_nan(float x, float y) {  // (a NaN stays one)
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// Weights of 16 rows from their scores `w`, in pairs: returned in `pw`.  `lift` holds the
// references' negatives; returns the largest exponent, NaN aside.
__device__ __forceinline__ float exponentials(const uint32_t (&w)[16], const float* qf, const float* lift, float ks,
                                              uint64_t (&pw)[8]) {
  const uint64_t ks2 = pack2(ks, ks);
  float over = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const ulonglong2 f = reinterpret_cast<const ulonglong2*>(qf)[i], m = reinterpret_cast<const ulonglong2*>(lift)[i];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = 4 * i + 2 * j;
      // (the factors first: their product with the sum is the score, so none is out of range before it)
      const float2 z = unpack2(fma2(pack2(__uint_as_float(w[e]), __uint_as_float(w[e + 1])), mul2(j ? f.y : f.x, ks2),
                                    j ? m.y : m.x));
      over = fmaxf(over, fmaxf(z.x, z.y));
      pw[2 * i + j] = pack2(fast_exp2(min_nan(z.x, kTop)), fast_exp2(min_nan(z.y, kTop)));
    }
  }
  return over;
}

// Weights times the token's value scale `vs`, as f16, to `row` (the token's row of P, swizzled
// by `sw`).  With kKeep a row that does not see the token has a product of 0 whatever `vs` is.
template <bool kKeep>
__device__ __forceinline__ void store_weights(const uint64_t (&pw)[8], float vs, uint32_t keep, uint4* row, int c, int sw) {
  const uint64_t vs2 = pack2(vs, vs);
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float2 x = unpack2(mul2(pw[i], vs2));
    if (kKeep) {
      if (!(keep >> (2 * i) & 1u)) x.x = 0.f;
      if (!(keep >> (2 * i + 1) & 1u)) x.y = 0.f;
    }
    const __half2 pr = __floats2half2_rn(x.x, x.y);
    h[i] = *reinterpret_cast<const uint32_t*>(&pr);
  }
  row[(2 * c) ^ sw] = make_uint4(h[0], h[1], h[2], h[3]);
  row[(2 * c + 1) ^ sw] = make_uint4(h[4], h[5], h[6], h[7]);
}

// A tile that some row may not see all of: scores times the key scale's fraction, -infinity for
// hidden ones, back to tensor memory (the caller goes on with the rest of the scale, which is a
// number above zero whatever the token's scale is).
__device__ __forceinline__ void hide(uint32_t tS, int nc, float ks, uint64_t keep) {
#pragma unroll 1
  for (int c = 0; c < nc; ++c, keep >>= 16) {
    uint32_t w[16];
    ld16(tS + 16 * c, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = uint32_t(keep) >> i & 1u ? __float_as_uint(__uint_as_float(w[i]) * ks) : 0xff800000u;
    tc::st16(tS + 16 * c, w);
  }
  tc::wait_st();
}

// Reduces 16 rows over the warpgroup's 128 tokens: every thread has its token's 16 values `x`;
// lane 2 r + (0 or 1) of each warp returns the result of row r.  (A warp's rows are halved as its
// lanes are: 16 shuffles for 16 rows.)  `part` is free when the warpgroup calls.
template <bool kMax>
__device__ __forceinline__ float reduce_rows(int id, int warp, int lane, float (&x)[16], float (*part)[16]) {
#pragma unroll
  for (int n = 8, o = 16; n > 0; n >>= 1, o >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      // (the upper lanes take the upper rows)
      const bool up = lane & o;
      const float mine = up ? x[n + i] : x[i], z = __shfl_xor_sync(0xffffffffu, up ? x[i] : x[n + i], o);
      x[i] = kMax ? fmaxf(mine, z) : mine + z;
    }
  const float z = __shfl_xor_sync(0xffffffffu, x[0], 1);
  const float y = kMax ? fmaxf(x[0], z) : x[0] + z;
  if (!(lane & 1)) part[warp][lane >> 1] = y;
  group_sync(id);
  const float* a = &part[0][lane >> 1];
  return kMax ? fmaxf(fmaxf(a[0], a[16]), fmaxf(a[32], a[48])) : (a[0] + a[16]) + (a[32] + a[48]);
}

// One key tile for the nc x 16 rows of a warpgroup.
//
// The weights are taken relative to the references as they are.  If one then turns out to
// exceed its reference by kGap the maxima are looked for, the references moved, and the tile's
// weights taken back and computed anew (a weight cut off at 2^kTop loses nothing: relative to the
// new reference the sum it was added to is below 2^-kTop).  An item's first tile starts there.
__device__ __forceinline__ void softmax_step(State* st, Rows& rw, const float* qf, const Token& tk, int nc, uint32_t tS,
                                             uint32_t tO, unsigned char* ptile, int c0, int step, bool first, Sums& l) {
  // (`ptile`: P, 64 rows of 128 tokens after another; `c0`: the warpgroup's first chunk of 16 rows)
  const int t = 32 * tk.warp + tk.lane;
  auto row = [&](int c) { return reinterpret_cast<uint4*>(ptile + ((c0 + c) >> 2) * (kBN * 128) + t * 128); };
  // (the product of the step before has read P)
  if (step > 0) (void)wait_warp(st, kODone + ((step - 1) & 1), uint32_t((step - 1) >> 1) & 1u);
  const float vs = tk.valid ? tk.vs : 0.f;
  if (!first) {
    float over = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
      uint32_t w[16];
      uint64_t pw[8];
      ld16(tS + 16 * c, w);
      over = fmaxf(over, exponentials(w, qf + 16 * c, rw.lift + 16 * c, tk.ks, pw));
      store_weights<false>(pw, vs, 0u, row(c), (c0 + c) & 3, t & 7);
      l.chunk(c, [&](uint64_t (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = add2(x[i], pw[i]);
      });
    }
    // (a value scale that is no number, and rows that must not meet it: the other way)
    if (!group_any(tk.id, over + tk.ex > kGap + i8::kTopWeight || (tk.cut && !(fabsf(vs) < INFINITY)))) return;
  }
  // the tile's maxima, row by row, and the new references
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    float x[16];
    {
      uint32_t w[16];
      float f[16];
      ld16(tS + 16 * c, w);
      lds16(qf + 16 * c, f);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = fmaf(__uint_as_float(w[i]), f[i] * tk.ks, tk.ex);
    }
    const float mx = reduce_rows<true>(tk.id, tk.warp, tk.lane, x, rw.part);
    if (tk.warp == 0 && !(tk.lane & 1)) {
      const int r = 16 * c + (tk.lane >> 1);
      const float m = rw.m[r];
      const bool go = mx > m + kGap || (m == -INFINITY && mx > -INFINITY);
      const float m2 = go ? mx : m;
      rw.m[r] = m2;
      rw.old[r] = first ? -INFINITY : rw.lift[r];
      rw.lift[r] = m2 == -INFINITY ? kNoLift : i8::kTopWeight - m2;
      rw.alpha[r] = go ? fast_exp2(m - m2) : 1.f;  // (0 from -infinity)
    }
    group_sync(tk.id);
  }
  tc::fence_after();  // (O^T holds the tiles before this one)
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    uint32_t w[16];
    uint64_t pw[8];
    ld16(tS + 16 * c, w);
    (void)exponentials(w, qf + 16 * c, rw.old + 16 * c, tk.ks, pw);
    const uint64_t minus = pack2(-1.f, -1.f);
    l.chunk(c, [&](uint64_t (&x)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fma2(pw[i], minus, x[i]);
    });
    ld16(tS + 16 * c, w);
    (void)exponentials(w, qf + 16 * c, rw.lift + 16 * c, tk.ks, pw);
    l.chunk(c, [&](uint64_t (&x)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fma2(x[i], reinterpret_cast<const uint64_t*>(rw.alpha + 16 * c)[i], pw[i]);
    });
    if (tk.cut)
      store_weights<true>(pw, vs, uint32_t(tk.keep >> (16 * c)), row(c), (c0 + c) & 3, t & 7);
    else
      store_weights<false>(pw, vs, 0u, row(c), (c0 + c) & 3, t & 7);
    if (first) continue;
    ld16(tO + 16 * c, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * rw.alpha[16 * c + i]);
    tc::st16(tO + 16 * c, w);
  }
  tc::wait_st();
}

// A warpgroup's query rows of an item (row0 .. row0 + half - 1) to f16, each scaled by a power
// of two of its own, and their score factors to `qf`.  `div`: 2^16 / group, rounded up.
template <int D>
__device__ __forceinline__ void load_queries(const TreeParams& p, const TreeSplit& sp, const Walk& it, const ItemRows& ir,
                                             int row0, unsigned char* q, float* qf, int warp, int lane,
                                             int div) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes, kBatch = 4;  // lanes of a row, rows of a pass, passes
  const int sub = lane / kLanes, col = (lane % kLanes) * 8, g = p.group;
  const int64_t tok0 = it.q.e.q0 + it.pair * sp.item_nodes;
#pragma unroll 1
  for (int i0 = warp * kBatch * kPer; i0 < ir.half; i0 += 4 * kBatch * kPer) {
    uint4 x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = row0 + i0 + u * kPer + sub;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < ir.rows) {
        const int node = (r * div) >> 16, h = r - node * g;  // (r < 256: exact)
        x[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.query) + (tok0 + node) * p.q_stride_t +
                                               int64_t(it.kvh * g + h) * p.q_stride_h + col);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kPer + sub, r = row0 + i;
      float f[8];
      Chunk<BF16>::expand(x[u], f);
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int sh = i8::query_shift(top);
      const float s = i8::power(sh), inv = i8::power(-sh);
      if (i < ir.half) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 v = __floats2half2_rn(f[2 * e] * s, f[2 * e + 1] * s);
          h[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(q + (col >> 6) * Cfg<D>::kQUnit + r * 128 + (((col >> 3) & 7) ^ (r & 7)) * 16) =
            make_uint4(h[0], h[1], h[2], h[3]);
        // (never 0, with which a hidden score of -infinity would be NaN)
        if (col == 0) qf[i] = fmaxf(p.qk_scale_log2 * inv, 0x1p-149f);
      }
    }
  }
}

// What write_rows needs of an item's part.
struct Part {
  int rows, tok0, kvh;  // query rows, their first node's, KV head
  bool whole, begins;
};

// Writes the rows' output, or the part of it, from O^T (lane = column of the head): a warp writes
// 32 columns of a row at a time.
template <int D>
__device__ __forceinline__ void write_rows(const TreeParams& p, const TreeSplit& sp, const Part& pt, Rows& rw, int id,
                                           int row0, int warp, int lane, int nc, uint32_t tO, int div, Sums& l) {
  const int64_t prow = int64_t(2 * blockIdx.x + (pt.begins ? 1 : 0)) * sp.rows;
  const int col = 32 * warp + lane;
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    float x[16];
    l.chunk(c, [&](uint64_t (&y)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 v = unpack2(y[i]);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
      }
    });
    const float sum = reduce_rows<false>(id, warp, lane, x, rw.part);
    if (warp == 0 && !(lane & 1)) {
      const int i = 16 * c + (lane >> 1), r = row0 + i;
      rw.alpha[i] = !pt.whole ? 1.f : sum != 0.f ? 1.f / sum : 0.f;
      if (!pt.whole && r < pt.rows) sp.ml[prow + r] = make_float2(rw.m[i], sum);
    }
    group_sync(id);
    uint32_t w[16];
    ld16(tO + 16 * c, w);
    if (col >= D) continue;  // (64 columns: the upper lanes of the accumulator repeat them)
    const int r0 = row0 + 16 * c, n = pt.rows - r0;
    if (pt.whole) {
      const int node = (r0 * div) >> 16;
      int h = r0 - node * p.group;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + int64_t(pt.tok0 + node) * p.out_stride_t +
                           int64_t(pt.kvh * p.group + h) * p.out_stride_h + col;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i < n) *out = __float2bfloat16_rn(__uint_as_float(w[i]) * rw.alpha[16 * c + i]);
        out += p.out_stride_h;
        if (++h == p.group) {
          h = 0;
          out += p.out_stride_t - p.group * p.out_stride_h;
        }
      }
    } else {
      float* o = sp.o + (prow + r0) * D + col;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) o[i * D] = __uint_as_float(w[i]) * rw.alpha[16 * c + i];
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tree_i8_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeSplit sp) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  State* st = reinterpret_cast<State*>(smem + C::kState);
  // (the warp's number from one lane: the compiler then knows that it is the same in all, and what
  // follows from it, a role's loops and addresses, is computed once for the warp)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int g = p.group;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      // one arrival per warp where a warpgroup arrives
      const bool warps4 = (i >= kCodeEmpty && i < kCodeEmpty + kMaxSlots) || (i >= kKFull && i < kKFull + 2) ||
                          (i >= kVFull && i < kVFull + 2);
      const bool warps8 = i == kQFull || (i >= kPFull && i < kPFull + 2) || (i >= kOFree && i < kOFree + 2);
      const bool lanes = i >= kScaleFull && i < kScaleFull + kScaleSlots;  // (each lane's copies)
      mbar_init(&st->bars[i], lanes ? 32 : warps8 ? 8 : warps4 ? 4 : 1);
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
  Walk it;
  it.start(p, sp, rg);

  // (each role takes its registers itself: the compiler counts them by branch)
  if (warp == 0 || warp == 3) {
    less_registers<kRegsControl>();
    // ---- codes, K by one warp and V by another, every second tile of the ring each: one bulk copy
    // per block of the cache (copies issued side by side from one warp go one by one, about 100
    // clocks each).  The first also copies the tokens' scales, four tokens to a lane ------------
    const int v = warp == 3, bs = p.block_size;
    const unsigned char* cache = static_cast<const unsigned char*>(v ? p.value_cache : p.key_cache);
    const uint32_t bytes = uint32_t(bs) * D;
    int slot = v, n = v;  // of the ring: tile and tile copies before this one
    uint32_t phase = 0;
    // tile j of `it` is looked up one tile before its copies are issued, over items too (up to
    // 64 blocks of two tokens: two to a lane)
    int j = it.valid() ? it.j0 : 0, kvh = 0, left = 0, nblk = 0, e0 = 0, e1 = 0;
    int tiles = 0, sslot = 0;  // of the scales' ring
    uint32_t sphase = 0;
    bool have = false;
    while (true) {
      const int kvh_now = kvh, left_now = left, nblk_now = nblk;
      int now[2] = {e0, e1};
      const bool copy = have;
      have = it.valid();
      if (have) {
        const int pos = it.q.base + j * kBN;
        kvh = it.kvh;
        left = max(0, min(kBN, it.q.e.L - pos));
        nblk = (left + bs - 1) >> sp.bs_shift;
        const int32_t* row = p.block_tables + int64_t(it.s) * p.bt_stride + (pos >> sp.bs_shift);
        e0 = lane < nblk ? __ldg(row + lane) : 0;
        e1 = lane + 32 < nblk ? __ldg(row + lane + 32) : 0;
        if (++j == it.j1) {
          it.next(p, sp, rg);
          j = it.j0;
        }
      }
      if (!copy) {
        if (!have) break;
        continue;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (now[u] < 0 || int64_t(now[u]) >= p.num_blocks) {
          raise_device_error(p.err, kErrTableEntry);
          now[u] = 0;
        }
      bool ok = true;
      if (n >= C::kSlots) ok = wait_warp(st, kCodeEmpty + slot, phase ^ 1u);
      if (ok) {
        if (lane == 0) mbar_arrive_expect_tx(&st->bars[kCodeFull + slot], uint32_t(nblk_now) * bytes);
        __syncwarp();
        unsigned char* dst = smem + C::kCodes + slot * C::kCodeBytes;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int b = lane + 32 * u;
          if (b < nblk_now)
            bulk_copy_g2s(dst + b * bytes, cache + int64_t(now[u]) * p.cs_block + int64_t(kvh_now) * p.cs_head, bytes,
                          &st->bars[kCodeFull + slot]);
        }
      }
      n += 2;
      slot += 2;
      if (slot >= C::kSlots) {
        slot -= C::kSlots;
        phase ^= 1u;
      }
      if (v) continue;
      // the tokens' scales: asynchronous copies of four tokens' 16 bytes where they are aligned
      // (their block's entry is in lane token / bs), else of each (the upper 32 blocks of two
      // tokens in the second register)
      if (tiles >= kScaleSlots) (void)wait_warp(st, kScaleEmpty + sslot, sphase ^ 1u);
      float* kd = &st->scales[sslot][0][4 * lane];
      float* vd = &st->scales[sslot][1][4 * lane];
      const int64_t head = int64_t(kvh_now) * p.ts_head;
      if (sp.vec_scales) {
        const int e = __shfl_sync(0xffffffffu, now[0], (4 * lane) >> sp.bs_shift);
        const bool there = 4 * lane < left_now;
        const int64_t at = there ? int64_t(e) * p.ts_block + head + ((4 * lane) & (bs - 1)) : 0;
        copy16(kd, p.k_token_scales + at, there);
        copy16(vd, p.v_token_scales + at, there);
      } else {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int b = (4 * lane + i) >> sp.bs_shift;
          const int ea = __shfl_sync(0xffffffffu, now[0], b & 31), eb = __shfl_sync(0xffffffffu, now[1], b & 31);
          const bool there = 4 * lane + i < left_now;
          const int64_t at = there ? int64_t(b < 32 ? ea : eb) * p.ts_block + head + ((4 * lane + i) & (bs - 1)) : 0;
          copy4(kd + i, p.k_token_scales + at, there);
          copy4(vd + i, p.v_token_scales + at, there);
        }
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_addr(&st->bars[kScaleFull + sslot]))
                   : "memory");
      ++tiles;
      if (++sslot == kScaleSlots) {
        sslot = 0;
        sphase ^= 1u;
      }
    }
    // the copies in flight land before the block may exit
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0)
      for (int k = max(0, n - C::kSlots); k < n; ++k)
        if ((k & 1) == v) (void)mbar_wait_bounded(&st->bars[kCodeFull + k % C::kSlots], uint32_t(k / C::kSlots) & 1u);
  } else if (warp == 1) {
    less_registers<kRegsControl>();
    // ---- score MMAs (a warp, see umma.cuh; the products' are another's: each waits only for its own) ----
    {
      const uint32_t base = smem_addr(smem);
      constexpr uint64_t kUnit = C::kUnitBytes >> 4;  // (descriptors hold addresses / 16)
      const uint64_t kdesc = tc::desc_sw128(base + C::kK, 16, 1024), qdesc = tc::desc_sw128(base + C::kQ, 16, 1024);
      int kn = 0, item = 0, n = 0;  // units of K, items, steps
      bool ok = true;
      for (; ok && it.valid(); it.next(p, sp, rg), ++item) {
        const ItemRows ir(p, sp, it);
        const uint32_t id = idesc_f16(kBN, ir.groups * ir.half, 0, 0);
        for (int j = it.j0; ok && j < it.j1; ++j, ++n) {
          if (j == it.j0) ok = wait_warp(st, kQFull, uint32_t(item) & 1u);
          // S^T and P of the step before last are free when its product is done (so the softmax
          // warps need not wait for that)
          if (n >= 2) ok = ok && wait_warp(st, kODone + (n & 1), uint32_t((n >> 1) - 1) & 1u);
          const uint32_t to = tmem + C::kS + (n & 1) * 128;
#pragma unroll 1
          for (int u = 0; ok && u < C::kUnits; ++u, ++kn) {
            if (!(ok = wait_warp(st, kKFull + (kn & 1), uint32_t(kn >> 1) & 1u))) break;
            tc::fence_after();
            const uint64_t kd = kdesc + (kn & 1) * kUnit, qd = qdesc + ((u * C::kQUnit) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) umma::mma_ss(to, kd + kk * 2, qd + kk * 2, id, (u > 0 || kk > 0) ? 1u : 0u);
            umma::commit(&st->bars[kKEmpty + (kn & 1)]);
          }
          if (ok) umma::commit(&st->bars[kSFull + (n & 1)]);
        }
      }
      // every MMA issued has completed before the tensor memory is freed
      umma::commit(&st->bars[kDrain]);
      (void)mbar_wait_bounded(&st->bars[kDrain], 0);
      if (!ok && lane == 0) raise_device_error(p.err, kErrTimeout);
    }
  } else if (warp == 2) {
    less_registers<kRegsControl>();
    // ---- product MMAs (a warp) -------------------------------------------------------------
    {
      const uint32_t base = smem_addr(smem);
      constexpr uint64_t kUnit = C::kUnitBytes >> 4;
      // (a head of 64 columns has one chunk of them: the second 64 rows of the MMA repeat it)
      const uint64_t vdesc = tc::desc_sw128(base + C::kV, D == 128 ? C::kVHalf : 0, 1024);
      const uint64_t pdesc = tc::desc_sw128(base + C::kP, C::kPBytes, 1024);
      int vn = 0, sslot = 0;  // units of V, the tile's slot of scales
      int n = 0, item = 0;  // steps, items
      int64_t at = rg->from;
      TreeSplit::Tail tail = {0, 0, 0, 0};  // what the fold needs of an item that goes on in the next range
      bool ok = true;
      for (; ok && it.valid(); it.next(p, sp, rg), ++item) {
        if (it.begins() && !it.ends()) {
          const int node0 = it.pair * sp.item_nodes;
          tail.row0 = it.q.e.q0 + node0;
          tail.nodes = min(sp.item_nodes, it.q.e.n - node0);
          tail.kvh = it.kvh;
          tail.last = int((at - it.u0 + it.q.tiles + rg->cost - 1) / rg->share);
        }
        at += it.u1 - it.u0;
        const ItemRows ir(p, sp, it);
        const uint32_t id = idesc_f16(128, ir.groups * ir.half, 1, 1);
        // (an O^T buffer is written again when the item before last has been written out)
        if (item >= 2) ok = wait_warp(st, kOFree + (item & 1), uint32_t((item >> 1) - 1) & 1u);
        const uint32_t to = tmem + C::kO + (item & 1) * 128;
        for (int j = it.j0; ok && j < it.j1; ++j, ++n) {
          ok = wait_warp(st, kPFull + (n & 1), uint32_t(n >> 1) & 1u);
#pragma unroll 1
          for (int u = 0; ok && u < C::kUnits; ++u, ++vn) {
            if (!(ok = wait_warp(st, kVFull + (vn & 1), uint32_t(vn >> 1) & 1u))) break;
            tc::fence_after();
            const uint64_t vd = vdesc + (vn & 1) * kUnit, pb = pdesc + ((u * C::kVTokens * 128) >> 4);
            const uint32_t acc = j > it.j0 || u > 0;
#pragma unroll
            for (int kk = 0; kk < C::kVTokens / 16; ++kk)
              umma::mma_ss(to, vd + kk * (16 * 128 >> 4), pb + kk * (16 * 128 >> 4), id, acc | (kk > 0));
            umma::commit(&st->bars[kVEmpty + (vn & 1)]);
          }
          if (!ok) break;
          umma::commit(&st->bars[kODone + (n & 1)]);
          umma::commit(&st->bars[kScaleEmpty + sslot]);  // (P, so the scales, have been used)
          if (++sslot == kScaleSlots) sslot = 0;
        }
      }
      if (lane == 0) sp.tails[blockIdx.x] = tail;
      umma::commit(&st->bars[kDrain + 1]);
      (void)mbar_wait_bounded(&st->bars[kDrain + 1], 0);
      if (!ok && lane == 0) raise_device_error(p.err, kErrTimeout);
    }
  } else if (warp >= 12) {
    less_registers<kRegsWiden>();
    // ---- widening: K by one warpgroup, V by the other, every second tile of the ring each -----
    const int v = warp >= 16, t = (tid - 384) & 127;
    // the thread's chunks of 16 codes of a unit: columns 16 (t % 4) .. of 64, rows t / 4 and 32
    // further ones (of a unit of V at D = 128: 32 further, then the other 64 columns)
    const int row = t >> 2, k = t & 3, sw = row & 7;
    const bool halves = v && D == 128;
    const uint32_t a = 32 * D, b = halves ? 64 : 64 * D, da = 32 * 128, db = halves ? C::kVHalf : 64 * 128;
    const unsigned char* src = smem + C::kCodes + row * D + k * 16;
    unsigned char* lo = smem + (v ? C::kV : C::kK) + row * 128 + ((2 * k ^ sw) << 4);
    unsigned char* hi = smem + (v ? C::kV : C::kK) + row * 128 + (((2 * k + 1) ^ sw) << 4);
    const int empty = v ? kVEmpty : kKEmpty, full = v ? kVFull : kKFull;
    const uint32_t unit_pitch = v ? C::kVTokens * D : 64;  // in the codes
    int slot = v, sslot = 0, n = 0;  // n: units
    uint32_t phase = 0, sphase = 0;
    for (; it.valid(); it.next(p, sp, rg)) {
      for (int j = it.j0; j < it.j1; ++j) {
        (void)wait_warp(st, kCodeFull + slot, phase);
        if (!v) {
          (void)wait_warp(st, kScaleFull + sslot, sphase);
          if (++sslot == kScaleSlots) {
            sslot = 0;
            sphase ^= 1u;
          }
        }
        const unsigned char* tile = src + slot * C::kCodeBytes;
#pragma unroll 1
        for (int u = 0; u < C::kUnits; ++u, ++n) {
          if (n > 1) (void)wait_warp(st, empty + (n & 1), uint32_t((n >> 1) - 1) & 1u);
          const uint32_t buf = (n & 1) * C::kUnitBytes;
          widen_unit(tile + u * unit_pitch, a, b, lo + buf, hi + buf, da, db);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (u == C::kUnits - 1) mbar_arrive(&st->bars[kCodeEmpty + slot]);
            mbar_arrive(&st->bars[full + (n & 1)]);
          }
        }
        slot += 2;
        if (slot >= C::kSlots) {
          slot -= C::kSlots;
          phase ^= 1u;
        }
      }
    }
  } else {
    more_registers<kRegsSoftmax>();
    // ---- softmax warpgroup `wg`: thread = token of the tile ---------------------------------
    const int wg = (warp >> 2) - 1, q = warp & 3, t = 32 * q + lane;
    const uint32_t lane_off = uint32_t(32 * q) << 16;
    Rows& rw = st->rows[wg];
    Token tk;
    tk.id = 1 + wg;
    tk.warp = q;
    tk.lane = lane;
    const int div = (65535 + g) / g;
    int item = 0, step = 0;
    // (Q is free once the scores of the item's last tile are there)
    auto queries = [&](const ItemRows& ir) {
      if (wg < ir.groups)
        load_queries<D>(p, sp, it, ir, wg * ir.half, smem + C::kQ, st->qf[item & 1][wg], q, lane, div);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&st->bars[kQFull]);
    };
    if (it.valid()) queries(ItemRows(p, sp, it));
    while (it.valid()) {
      const ItemRows ir(p, sp, it);
      const int row0 = wg * ir.half, nc = wg < ir.groups ? ir.half >> 4 : 0, ob = item & 1;
      {
        const Extent& e = it.q.e;
        const uint32_t tO = tmem + C::kO + ob * 128 + row0 + lane_off;
        const float* qf = st->qf[item & 1][wg];
        Sums l;
#pragma unroll
        for (int i = 0; i < kHalfRows / 2; ++i) l.a[i >> 3][i & 7] = 0ull;
        if (t < kHalfRows) {
          rw.m[t] = -INFINITY;
          rw.lift[t] = kNoLift;
        }
        group_sync(tk.id);
#pragma unroll 1
        for (int j = it.j0; j < it.j1; ++j, ++step) {
          const int pos = it.q.base + j * kBN + t;
          tk.valid = pos >= e.lo && pos < e.L;
          tk.cut = it.cut(j);
          tk.keep = ~0ull;
          if (tk.cut) {
            if (!tk.valid) {
              tk.keep = 0;
            } else if (p.tree_mask && pos >= e.P) {
              // the rows (node by node, g each) that see this node
              const int c = pos - e.P, r0 = row0;
              tk.keep = 0;
              int node = r0 / g, h = r0 - node * g;
              const int64_t* mask = p.tree_mask + (e.q0 + it.pair * sp.item_nodes + node) * p.mask_stride;
              for (int r = r0; r < min(ir.rows, r0 + ir.half);) {
                const int len = g - h;  // rows left of the node
                if (sees_node(mask, c)) {
                  const int at = r - r0;
                  tk.keep |= (len >= 64 ? ~0ull : (1ull << len) - 1) << at;
                }
                r += len;
                h = 0;
                mask += p.mask_stride;
              }
            }
          }
          (void)wait_warp(st, kSFull + (step & 1), uint32_t(step >> 1) & 1u);
          tc::fence_after();
          const int sl = step % kScaleSlots;  // (the tile's scales are there: its K waited for them)
          tk.ks = st->scales[sl][0][t];
          tk.vs = st->scales[sl][1][t];
          tk.ex = i8::scale_exponent(tk.vs);
          const uint32_t tS = tmem + C::kS + (step & 1) * 128 + row0 + lane_off;
          if (tk.cut) {
            // (a power of two of it is left for later: a sum times all of it may be out of range)
            const int ke = max(0, min(126, int(__float_as_uint(fabsf(tk.ks)) >> 23) - 127));
            hide(tS, nc, tk.ks * i8::power(-ke), tk.keep);
            tk.ks = i8::power(ke);
          }
          const bool first = j == it.j0;
          if (nc > 0)
            softmax_step(st, rw, qf, tk, nc, tS, tO, smem + C::kP, row0 >> 4, step, first, l);
          fence_proxy_async_smem();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&st->bars[kPFull + (step & 1)]);
        }
        const Part pt = {ir.rows, e.q0 + it.pair * sp.item_nodes, it.kvh, it.begins() && it.ends(), it.begins()};
        it.next(p, sp, rg);
        ++item;
        if (it.valid()) queries(ItemRows(p, sp, it));  // (the next item's scores, while this one is written)
        (void)wait_warp(st, kODone + ((step - 1) & 1), uint32_t((step - 1) >> 1) & 1u);
        tc::fence_after();
        write_rows<D>(p, sp, pt, rw, tk.id, row0, q, lane, nc, tO, div, l);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->bars[kOFree + ob]);
      }
    }
    if (lane == 0 && st->abort) raise_device_error(p.err, kErrTimeout);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(tmem, kTmemCols);
}

}  // namespace tree_i8

namespace {

template <int D>
cudaError_t launch_tree_i8_tpl(const TreeParams& p, const TreeSplit& sp, cudaStream_t stream) {
  using C = tree_i8::Cfg<D>;
  static_assert(sizeof(tree_i8::State) <= C::kStateBytes, "state");
  static_assert(C::kSmem <= 227 * 1024, "shared memory");
  static_assert(C::kSlots >= 2 && C::kSlots <= tree_i8::kMaxSlots, "ring");
  constexpr int kDevices = 64;
  auto kern = tree_i8::tree_i8_kernel<D>;
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
  cfg.blockDim = dim3(tree_i8::kThreads);
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

bool tree_i8_supported(const TreeParams& p) {
  if (p.q_dtype != kBF16 || p.kv_dtype != kI8) return false;
  if (p.group > tree::kBM) return false;
  if (!(p.qk_scale_log2 > 0.f)) return false;  // (limits are divided by the row's factor)
  if ((reinterpret_cast<uintptr_t>(p.query) & 15) || (p.q_stride_t & 7) || (p.q_stride_h & 7)) return false;
  return true;
}

cudaError_t launch_tree_i8(const TreeParams& p, TreeSplit sp, cudaStream_t stream) {
  sp.item_nodes = sp.tq;
  sp.vec_scales = p.block_size >= 4 && !((reinterpret_cast<uintptr_t>(p.k_token_scales) |
                                          reinterpret_cast<uintptr_t>(p.v_token_scales)) & 15) &&
                  !(p.ts_block & 3) && !(p.ts_head & 3);
  return p.head_dim == 128 ? launch_tree_i8_tpl<128>(p, sp, stream) : launch_tree_i8_tpl<64>(p, sp, stream);
}

}  // namespace pkv
