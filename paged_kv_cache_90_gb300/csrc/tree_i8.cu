// tree_i8.cu — decode attention and attention of drafted trees over a token-scaled int8
// cache on the fifth-generation tensor cores.
//
// A cached token is head_dim codes and one scale.  With the MMA's 128 rows on the tokens of a
// key tile and its columns on the query rows (drafted nodes x the group's heads, up to 128),
// a token's two scales belong to one thread, the work of a softmax grows with the rows that
// there are, and few rows cost little:
//   S^T = K Q^T         M = 128 tokens, N = rows, K = D: K codes widened to f16 and Q (f16) in
//                       shared memory, S^T in tensor memory, lane = token
//   P^T = 2^(S ks c - m) vs   by one thread per token, written to shared memory as f16
//   O^T += V^T P^T      M = D, N = rows, K = 128 tokens: V codes widened to f16, O^T in
//                       tensor memory, lane = column of the head
// The rows go in two halves to two softmax warpgroups (one, if there are at most 16), each with
// its own P, S^T buffers and O^T; every key tile is widened once for all of them.
//
// The codes are whole numbers, so f16 holds them exactly; a query row is scaled by a power of
// two that brings its largest element to 2^14, so its bf16 values are exact down to 2^-29 of
// that.  A weight times its value scale is rounded to f16 (half a step, 2^-11), relative to the
// running largest value scale, a power of two; maximum, sum, scores and output stay in binary32.
// A row's reference maximum moves when a score exceeds it by 2^8, the value scales' when one
// exceeds it by 2^4: whether any thread of the warpgroup saw one is one barrier per tile, and
// only then are the maxima looked for.
//
// A tile is 2 x 128 x (D + 4) bytes from HBM, and 2 x 128 x D codes to widen: about 27 warp
// instructions for 512 codes (an exclusive-or, two byte permutes and two subtractions for four
// codes), one warpgroup's whole work.  HBM bounds the long calls as long as enough copies are
// in flight; shared memory (codes in and out, operands in, and read by two MMAs: 176 KB per
// 32 KB tile at D = 128) is close behind.
//
// Warps: 0 streams codes, K and V tiles in turn (bulk copies of one (block, head) run each); 1
// issues the MMAs; 3 the queries; 4-7 and 8-11 are the softmax warpgroups; 12-15 widen K, 16-19 V.  Every
// wait is bounded; when one runs out the block sets an error bit and a flag, every role runs
// through its loops without waiting, lets its copies and MMAs land and frees the tensor memory.
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "tcgen05.cuh"
#include "tree_split.cuh"

namespace pkv {
namespace tree_i8 {

using namespace tree;

constexpr int kThreads = 640;
// registers of a thread, by warpgroup: launched with 96 each (5 x 96 = 480), then split anew
// into control, two softmax and two widening warpgroups (80 + 2 x 144 + 2 x 56 = 480)
constexpr int kRegsControl = 80, kRegsSoftmax = 144, kRegsWiden = 56;
static_assert(kRegsControl + 2 * kRegsSoftmax + 2 * kRegsWiden <= 5 * 96, "registers");
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxSlots = 16;  // of the ring of code tiles
constexpr int kFewRows = 16;   // rows that one warpgroup takes alone
constexpr int kHalfRows = 64;  // rows of a warpgroup at most

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kHalfBytes = kBN * 128;  // one 64-column half of an operand tile
  static constexpr uint32_t kOpBytes = kHalves * kHalfBytes;
  static constexpr uint32_t kCodeBytes = kBN * D;
  static constexpr uint32_t kPBytes = kBN * 128;
  // from the 1024-aligned base: widened K | widened V | Q | P | ring of code tiles | state.  A
  // batch of few rows needs one P and 16 rows of Q, and the ring has the rest.
  static constexpr uint32_t kK = 0, kV = kOpBytes, kQ = 2 * kOpBytes;
  static constexpr uint32_t kState = 212 * 1024;
  static constexpr uint32_t kStateBytes = 10 * 1024;
  static constexpr size_t kSmem = kState + kStateBytes + 1024;  // (+ alignment)
  // tensor memory: S^T [warpgroup][2], then O^T [2][warpgroup], 64 columns each
  static constexpr uint32_t kS = 0, kO = 256;
};

enum Bar { kQFull = 0, kQEmpty, kCodeFull, kCodeEmpty = kCodeFull + kMaxSlots, kKFull = kCodeEmpty + kMaxSlots, kKEmpty,
           kVFull, kVEmpty, kSFull, kPFull = kSFull + 4, kODone = kPFull + 2, kOFree = kODone + 2, kDrain = kOFree + 4,
           kNumBars };

// What a warpgroup keeps of its rows.
struct Rows {
  float m[kHalfRows];        // reference maximum (base 2), -infinity before the first score
  float limit[kHalfRows];    // a score before its row's factor above this moves it
  float shift[kHalfRows];    // m, or 0 where it is -infinity
  float alpha_l[kHalfRows];  // the last move's factors on the sums and on the output
  float alpha_o[kHalfRows];
  float part[4][kHalfRows];  // per warp: maxima on the way, sums at the end
  float vpart[4];
};

struct State {
  uint64_t bars[kNumBars + 1];
  volatile int abort;
  uint32_t tmem;
  Range range;
  longlong2 warp_sum[kThreads / 32];
  float qf[4][2][kHalfRows];  // a row's score factor, per item (index mod 4: a warpgroup may be
                              // two items behind the queries)
  Rows rows[2];
};

// A wait that runs out tells the others and is not one for the loops to stop at: a role
// whose waits fail runs through its loops, so that barriers among warps always meet.
__device__ __forceinline__ bool wait(State* st, int bar, uint32_t parity) {
  if (mbar_try_wait(&st->bars[bar], parity)) return true;
  return !st->abort && tree::wait(&st->bars[bar], parity, &st->abort);
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

// Four int8 codes -> four f16 values, exact: code + 128 in the low byte of 0x64.. is 1152 +
// code in f16.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), off), y = __hsub2(*reinterpret_cast<__half2*>(&b), off);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// A tile of codes [128][D] -> f16 operand tile (128-byte rows of 64 columns, swizzled), by
// the 128 threads of a widening warpgroup.  `src` and `dst` are the thread's first chunk of 16
// codes and its row: the next one is 2048 / D rows, a multiple of 8, further (so the swizzle
// stays).
template <int D>
__device__ __forceinline__ void widen_tile(const unsigned char* src, unsigned char* dst, uint32_t at0, uint32_t at1,
                                           bool swap) {
  constexpr int kChunks = kBN * D / 16 / 128, kRows = 128 * 16 / D;
#pragma unroll 2
  for (int i = 0; i < kChunks; ++i) {
    const uint4 c = *reinterpret_cast<const uint4*>(src + i * 2048);
    const uint2 a = widen4(c.x), b = widen4(c.y), e = widen4(c.z), f = widen4(c.w);
    const uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(e.x, e.y, f.x, f.y);
    // (the upper half's chunks go in the other order: no two lanes on one bank)
    *reinterpret_cast<uint4*>(dst + i * kRows * 128 + at0) = swap ? hi : lo;
    *reinterpret_cast<uint4*>(dst + i * kRows * 128 + at1) = swap ? lo : hi;
  }
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

// Largest of a warp's values, NaN aside (an order-preserving map to integers).
__device__ __forceinline__ float warp_max(float x) {
  const int i = __float_as_int(x == x ? x : -INFINITY);
  const int o = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7fffffff));
  return __int_as_float(o ^ ((o >> 31) & 0x7fffffff));
}

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

// A softmax warpgroup's thread: token `t` of the tile, its rows' sums in registers.
struct Token {
  int id;          // the warpgroup's barrier
  int warp, lane;  // of the warpgroup
  float ks, vs;    // the token's scales
  bool valid;      // the token is a position of the row's range
  bool cut;        // some row may not see it: `keep` says which do
  uint64_t keep;
};

// The sums of a thread's rows, 16 to an array so that loops over the rows need no unrolling
// (unrolled code misses the instruction cache at every tile): a register array takes constant
// indices only.
struct Sums {
  float a[4][16];
  template <typename F>
  __device__ __forceinline__ void chunk(int c, F f) {
    if (c == 0) f(a[0]);
    else if (c == 1) f(a[1]);
    else if (c == 2) f(a[2]);
    else f(a[3]);
  }
};

// Weights of the 16 rows at tensor-memory column `ts`: added to their sums, and times the
// token's value scale `vn` written as f16 to `row` (the token's row of P, swizzled by `sw`).
template <bool kCut>
__device__ __forceinline__ void weights(uint32_t ts, const float* qf, const float* shift, float ks, float vn,
                                        uint32_t keep, float (&pw)[16], uint4* row, int c, int sw) {
  uint32_t w[16], h[8];
  float f[16], sh[16];
  ld16(ts, w);
  lds16(qf, f);
  lds16(shift, sh);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    pw[i] = fast_exp2(fmaf(__uint_as_float(w[i]) * ks, f[i], -sh[i]));
    pw[i + 1] = fast_exp2(fmaf(__uint_as_float(w[i + 1]) * ks, f[i + 1], -sh[i + 1]));
    float a = pw[i] * vn, b = pw[i + 1] * vn;
    if (kCut) {  // (a position that is not seen has weight 0 whatever its scales are)
      if (!(keep >> i & 1u)) pw[i] = a = 0.f;
      if (!(keep >> (i + 1) & 1u)) pw[i + 1] = b = 0.f;
    }
    const __half2 pr = __floats2half2_rn(a, b);
    h[i / 2] = *reinterpret_cast<const uint32_t*>(&pr);
  }
  row[(2 * c) ^ sw] = make_uint4(h[0], h[1], h[2], h[3]);
  row[(2 * c + 1) ^ sw] = make_uint4(h[4], h[5], h[6], h[7]);
}

// One key tile for the nc x 16 rows of a warpgroup.  `vref`: the power of two that value
// scales are taken relative to (0 at first).
__device__ __forceinline__ void softmax_step(State* st, Rows& rw, const float* qf, const Token& tk, int nc, uint32_t tS,
                                             uint32_t tO, unsigned char* ptile, int done_bar, int step, bool first,
                                             float& vref, Sums& l) {
  const int t = 32 * tk.warp + tk.lane;
  // does a score, or the value scale, exceed its reference?
  const float av = fabsf(tk.vs);
  bool move = tk.valid && av > 16.f * vref && av < INFINITY;
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    uint32_t w[16];
    float lim[16];
    ld16(tS + 16 * c, w);
    lds16(rw.limit + 16 * c, lim);
    uint32_t over = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) over |= __uint_as_float(w[i]) * tk.ks > lim[i] ? 1u << i : 0u;
    if (tk.cut) over &= uint32_t(tk.keep >> (16 * c));
    move |= (over & 0xffffu) != 0u;
  }
  if (group_any(tk.id, move)) {
    // the tile's maxima, row by row, and the new references
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
      uint32_t w[16];
      float f[16];
      ld16(tS + 16 * c, w);
      lds16(qf + 16 * c, f);
      const uint32_t kp = uint32_t(tk.keep >> (16 * c));
      float mine = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float z = warp_max(kp >> i & 1u ? __uint_as_float(w[i]) * tk.ks * f[i] : -INFINITY);
        if (tk.lane == i) mine = z;
      }
      if (tk.lane < 16) rw.part[tk.warp][16 * c + tk.lane] = mine;
    }
    const float wv = warp_max(tk.valid && av < INFINITY ? av : 0.f);
    if (tk.lane == 0) rw.vpart[tk.warp] = wv;
    group_sync(tk.id);
    const float top = fmaxf(fmaxf(rw.vpart[0], rw.vpart[1]), fmaxf(rw.vpart[2], rw.vpart[3]));
    float valpha = 1.f;
    if (top > 16.f * vref) {
      // the power of two at or above it (subnormal ones: the smallest normal)
      const uint32_t b = __float_as_uint(fmaxf(top, 0x1p-126f));
      const float up = __uint_as_float((b & 0x7f800000u) + ((b & 0x7fffffu) ? 0x800000u : 0u));
      const float ref = fminf(up, 0x1p127f);
      valpha = vref / ref;  // (both powers of two, or 0)
      vref = ref;
    }
    if (t < 16 * nc) {
      const float mx = fmaxf(fmaxf(rw.part[0][t], rw.part[1][t]), fmaxf(rw.part[2][t], rw.part[3][t]));
      const float m = rw.m[t];
      const bool go = mx > m + kGap || (m == -INFINITY && mx > -INFINITY);
      const float m2 = go ? mx : m;
      const float a = go ? fast_exp2(m - m2) : 1.f;  // (0 from -infinity)
      rw.m[t] = m2;
      rw.limit[t] = (m2 + kGap) / qf[t];  // (a row's factor is above zero)
      rw.shift[t] = m2 == -INFINITY ? 0.f : m2;
      rw.alpha_l[t] = a;
      rw.alpha_o[t] = a * valpha;
    }
    group_sync(tk.id);
    if (!first) {
      // O^T holds the tiles before this one
      (void)__all_sync(0xffffffffu, wait(st, done_bar, uint32_t(step - 1) & 1u));
      tc::fence_after();
#pragma unroll 1
      for (int c = 0; c < nc; ++c) {
        uint32_t w[16];
        float a[16];
        lds16(rw.alpha_l + 16 * c, a);
        l.chunk(c, [&](float (&x)[16]) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= a[i];
        });
        ld16(tO + 16 * c, w);
        lds16(rw.alpha_o + 16 * c, a);
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * a[i]);
        tc::st16(tO + 16 * c, w);
      }
      tc::wait_st();
    }
  }
  // the weights (P's last product has to be done before its tile is written again)
  if (step > 0) (void)__all_sync(0xffffffffu, wait(st, done_bar, uint32_t(step - 1) & 1u));
  const float vn = tk.valid ? tk.vs * (vref > 0.f ? 1.f / vref : 0.f) : 0.f;
  uint4* row = reinterpret_cast<uint4*>(ptile + t * 128);
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    float pw[16];
    if (tk.cut)
      weights<true>(tS + 16 * c, qf + 16 * c, rw.shift + 16 * c, tk.ks, vn, uint32_t(tk.keep >> (16 * c)), pw, row, c, t & 7);
    else
      weights<false>(tS + 16 * c, qf + 16 * c, rw.shift + 16 * c, tk.ks, vn, 0u, pw, row, c, t & 7);
    l.chunk(c, [&](float (&x)[16]) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] += pw[i];
    });
  }
}

// Writes the rows' output, or the part of it, from O^T.
template <int D>
__device__ __forceinline__ void write_rows(const TreeParams& p, const TreeSplit& sp, const Walk& it, const ItemRows& ir,
                                           Rows& rw, int id, int wg, int warp, int lane, int nc, uint32_t tO, float vref,
                                           Sums& l) {
  const int row0 = wg * ir.half, t = 32 * warp + lane;
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    float x[16];
    l.chunk(c, [&](float (&y)[16]) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = y[i];
    });
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
      if (lane == 0) rw.part[warp][16 * c + i] = x[i];
    }
  }
  group_sync(id);
  const bool whole = it.begins() && it.ends();
  const int64_t prow = int64_t(2 * blockIdx.x + (it.begins() ? 1 : 0)) * sp.rows + row0;
  if (t < 16 * nc) {
    const float sum = (rw.part[0][t] + rw.part[1][t]) + (rw.part[2][t] + rw.part[3][t]);
    rw.alpha_o[t] = whole ? (sum != 0.f ? vref / sum : 0.f) : vref;
    if (!whole && row0 + t < ir.rows) sp.ml[prow + t] = make_float2(rw.m[t], sum);
  }
  group_sync(id);
  const int64_t tok0 = it.q.e.q0 + it.pair * sp.item_nodes;
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    uint32_t w[16];
    float a[16];
    ld16(tO + 16 * c, w);
    if (t >= D) continue;  // (64 columns: the upper lanes repeat them)
    lds16(rw.alpha_o + 16 * c, a);
    const int r0 = row0 + 16 * c, n = min(16, ir.rows - r0);
    int node = r0 / p.group, h = r0 - node * p.group;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i < n) {
        const float v = __uint_as_float(w[i]) * a[i];
        if (whole)
          static_cast<__nv_bfloat16*>(p.out)[(tok0 + node) * p.out_stride_t +
                                             int64_t(it.kvh * p.group + h) * p.out_stride_h + t] = __float2bfloat16_rn(v);
        else
          sp.o[(prow + 16 * c + i) * D + t] = v;
        if (++h == p.group) {
          h = 0;
          ++node;
        }
      }
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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = p.group;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      // one arrival per warp where a warpgroup arrives
      const bool warps4 = (i >= kCodeEmpty && i < kCodeEmpty + kMaxSlots) || i == kKFull || i == kVFull ||
                          (i >= kPFull && i < kPFull + 2) || (i >= kOFree && i < kOFree + 4);
      mbar_init(&st->bars[i], warps4 ? 4 : 1);
    }
    st->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) tc::alloc(&st->tmem, kTmemCols);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing of the caller's is read before
  asm volatile("griddepcontrol.launch_dependents;");
  const bool many = find_range<kThreads>(p, sp, &st->range, st->warp_sum, kFewRows / g);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = st->tmem;
  const Range* rg = &st->range;
  Walk it;
  it.start(p, sp, rg);
  // the layout behind the widened tiles
  const int q_rows = many ? kHalfRows : kFewRows, groups = many ? 2 : 1;  // of Q, per warpgroup
  const uint32_t q_half = uint32_t(q_rows) * 128, q_group = q_half * C::kHalves;
  const uint32_t oP = C::kQ + groups * q_group, oCodes = oP + groups * C::kPBytes;
  const int slots = min(kMaxSlots, int((C::kState - oCodes) / C::kCodeBytes));  // (K and V in turn, odd or even)

  // (each role takes its registers itself: the compiler counts them by branch)
  if (warp == 0) {
    less_registers<kRegsControl>();
    // ---- codes: K then V of every tile, one bulk copy per block of the cache ----------------
    const int bs = p.block_size;
    const uint32_t bytes = uint32_t(bs) * D;
    int slot = 0, n = 0;
    uint32_t phase = 0;
    for (; it.valid(); it.next(p, sp, rg)) {
      const int32_t* row = p.block_tables + int64_t(it.s) * p.bt_stride;
      for (int j = it.j0; j < it.j1; ++j) {
        const int pos = it.q.base + j * kBN;
        const int nblk = (max(0, min(kBN, it.q.e.L - pos)) + bs - 1) >> sp.bs_shift;
        // (up to 64 blocks of two tokens: two to a lane)
        int e[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int b = lane + 32 * u;
          e[u] = 0;
          if (b < nblk) {
            e[u] = __ldg(row + (pos >> sp.bs_shift) + b);
            if (e[u] < 0 || int64_t(e[u]) >= p.num_blocks) {
              raise_device_error(p.err, kErrTableEntry);
              e[u] = 0;
            }
          }
        }
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          bool ok = true;
          if (lane == 0 && n >= slots) ok = wait(st, kCodeEmpty + slot, phase ^ 1u);
          ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
          if (ok) {
            if (lane == 0) mbar_arrive_expect_tx(&st->bars[kCodeFull + slot], uint32_t(nblk) * bytes);
            __syncwarp();
            const unsigned char* src = static_cast<const unsigned char*>(v ? p.value_cache : p.key_cache);
            unsigned char* dst = smem + oCodes + slot * C::kCodeBytes;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int b = lane + 32 * u;
              if (b < nblk)
                bulk_copy_g2s(dst + b * bytes, src + int64_t(e[u]) * p.cs_block + int64_t(it.kvh) * p.cs_head, bytes,
                              &st->bars[kCodeFull + slot]);
            }
            ++n;
            if (++slot == slots) {
              slot = 0;
              phase ^= 1u;
            }
          }
        }
      }
    }
    // the copies in flight land before the block may exit
    if (lane == 0)
      for (int k = max(0, n - slots); k < n; ++k)
        (void)mbar_wait_bounded(&st->bars[kCodeFull + k % slots], uint32_t(k / slots) & 1u);
  } else if (warp == 1) {
    less_registers<kRegsControl>();
    // ---- MMAs (one thread): scores run up to two tiles ahead of the products ----------------
    if (lane == 0) {
      const uint32_t base = smem_addr(smem);
      const uint64_t kdesc = tc::desc_sw128(base + C::kK, 16, 1024);
      // (a head of 64 columns has one chunk of them: the second 64 rows of the MMA repeat it)
      const uint64_t vdesc = tc::desc_sw128(base + C::kV, D == 128 ? C::kHalfBytes : 0, 1024);
      const uint64_t qdesc = tc::desc_sw128(base + C::kQ, 16, 1024), pdesc = tc::desc_sw128(base + oP, 16, 1024);
      struct Pending {
        int half;
        bool two, first;
        uint8_t ob, of;  // O^T buffers of the two groups (bits), and whether they are waited for and the phases
        uint8_t wait;
      };
      Pending pend[2];
      int ts = 0, tp = 0;            // tiles whose scores, and products, have been issued
      int done = 0;                  // groups of tile tp whose product has been issued
      int j = it.j0, item = 0;
      int use[2] = {0, 0};           // items of the warpgroups so far (constant indices: registers)
      int sn0 = 0, sn1 = 0, pn0 = 0, pn1 = 0;  // their steps
      uint32_t idle = 0;
      bool ok = true;
      while (it.valid() || tp < ts) {
        bool went = false;
        if (it.valid() && ts <= tp + 1 && test_wait(&st->bars[kKFull], uint32_t(ts) & 1u) &&
            (j > it.j0 || test_wait(&st->bars[kQFull], uint32_t(item) & 1u))) {
          tc::fence_after();
          const ItemRows ir(p, sp, it);
          const uint32_t id = idesc_f16(kBN, ir.half, 0, 0);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (w < ir.groups) {
              const int n = w ? sn1 : sn0;
              const uint32_t ts_col = tmem + C::kS + w * 128 + (n & 1) * 64;
              const uint64_t qd = qdesc + (w * q_group >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc::mma_ss(ts_col, kdesc + ((kk >> 2) * C::kHalfBytes >> 4) + (kk & 3) * 2,
                           qd + ((kk >> 2) * q_half >> 4) + (kk & 3) * 2, id, kk > 0 ? 1u : 0u);
              tc::commit(&st->bars[kSFull + 2 * w + (n & 1)]);
            }
          }
          tc::commit(&st->bars[kKEmpty]);
          if (j == it.j1 - 1) tc::commit(&st->bars[kQEmpty]);
          Pending pd;
          pd.half = ir.half;
          pd.two = ir.groups == 2;
          pd.first = j == it.j0;
          pd.ob = uint8_t((use[0] & 1) | (use[1] & 1) << 1);
          pd.wait = uint8_t((use[0] >= 2 ? 1 : 0) | (use[1] >= 2 ? 2 : 0));
          pd.of = uint8_t((((use[0] - 2) >> 1) & 1) | (((use[1] - 2) >> 1) & 1) << 1);
          if (ts & 1) pend[1] = pd; else pend[0] = pd;
          ++ts;
          ++sn0;
          if (pd.two) ++sn1;
          if (++j == it.j1) {
            ++use[0];
            if (pd.two) ++use[1];
            ++item;
            it.next(p, sp, rg);
            j = it.j0;
          }
          went = true;
        }
        if (tp < ts) {
          const Pending pd = (tp & 1) ? pend[1] : pend[0];
          const int w = done, n = w ? pn1 : pn0, ob = (pd.ob >> w) & 1;
          if (test_wait(&st->bars[kPFull + w], uint32_t(n) & 1u) && test_wait(&st->bars[kVFull], uint32_t(tp) & 1u) &&
              (!pd.first || !((pd.wait >> w) & 1) || test_wait(&st->bars[kOFree + 2 * w + ob], (pd.of >> w) & 1u))) {
            tc::fence_after();
            const uint32_t id = idesc_f16(128, pd.half, 1, 1);
            const uint32_t to = tmem + C::kO + ob * 128 + w * 64;
            const uint64_t pdsc = pdesc + (w * C::kPBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk)
              tc::mma_ss(to, vdesc + kk * (16 * 128 >> 4), pdsc + kk * (16 * 128 >> 4), id,
                         (!pd.first || kk > 0) ? 1u : 0u);
            tc::commit(&st->bars[kODone + w]);
            if (w) ++pn1; else ++pn0;
            if (++done == (pd.two ? 2 : 1)) {
              tc::commit(&st->bars[kVEmpty]);
              done = 0;
              ++tp;
            }
            went = true;
          }
        }
        if (went) {
          idle = 0;
        } else {
          __nanosleep(20);
          if ((++idle & 255u) == 0 && (st->abort || idle > kWaitPolls)) {
            ok = false;
            break;
          }
        }
      }
      // every MMA issued has completed before the tensor memory is freed
      tc::commit(&st->bars[kDrain]);
      (void)mbar_wait_bounded(&st->bars[kDrain], 0);
      if (!ok) {
        st->abort = 1;
        raise_device_error(p.err, kErrTimeout);
      }
    }
  } else if (warp == 2) {
    less_registers<kRegsControl>();
  } else if (warp == 3) {
    less_registers<kRegsControl>();
    // ---- queries: an item's rows to f16, each scaled by a power of two of its own; and what
    // the fold needs of an item that goes on in the next block's range ------------------------
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a row, rows of a pass
    const int sub = lane / kLanes, col = (lane % kLanes) * 8;
    int item = 0;
    int64_t at = rg->from;
    TreeSplit::Tail tail = {0, 0, 0, 0};
    for (; it.valid(); it.next(p, sp, rg), ++item) {
      const ItemRows ir(p, sp, it);
      const int node0 = it.pair * sp.item_nodes;
      const int64_t tok0 = it.q.e.q0 + node0;
      if (item > 0) (void)__all_sync(0xffffffffu, wait(st, kQEmpty, uint32_t(item - 1) & 1u));
      constexpr int kBatch = 8;
      for (int r0 = 0; r0 < ir.groups * ir.half; r0 += kBatch * kPer) {
        uint4 x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int r = r0 + u * kPer + sub;
          x[u] = make_uint4(0u, 0u, 0u, 0u);
          if (r < ir.rows) {
            const int node = r / g, h = r - node * g;
            x[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.query) + (tok0 + node) * p.q_stride_t +
                                                   int64_t(it.kvh * g + h) * p.q_stride_h + col);
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int r = r0 + u * kPer + sub;
          float f[8];
          Chunk<BF16>::expand(x[u], f);
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          // 2^(14 - exponent of the largest), kept within 2^-100 .. 2^100
          const int ex = int(__float_as_uint(top) >> 23) - 127;
          const int sh = top > 0.f && top < INFINITY ? max(-100, min(100, 14 - ex)) : 0;
          const float s = __uint_as_float(uint32_t(127 + sh) << 23), inv = __uint_as_float(uint32_t(127 - sh) << 23);
          if (r < ir.groups * ir.half) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __half2 v = __floats2half2_rn(f[2 * i] * s, f[2 * i + 1] * s);
              h[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            const int w = r >= ir.half, n = r - w * ir.half;
            unsigned char* q = smem + C::kQ + w * q_group + (col >> 6) * q_half + n * 128;
            *reinterpret_cast<uint4*>(q + (((col >> 3) & 7) ^ (n & 7)) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
            if (col == 0) st->qf[item & 3][w][n] = p.qk_scale_log2 * inv;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&st->bars[kQFull]);
      if (it.begins() && !it.ends()) {
        tail.row0 = int(tok0);
        tail.nodes = min(sp.item_nodes, it.q.e.n - node0);
        tail.kvh = it.kvh;
        tail.last = int((at - it.u0 + it.q.tiles + rg->cost - 1) / rg->share);
      }
      at += it.u1 - it.u0;
    }
    if (lane == 0) sp.tails[blockIdx.x] = tail;
  } else if (warp >= 12) {
    less_registers<kRegsWiden>();
    // ---- widening: K by one warpgroup, V by the other, every second tile of the ring each -----
    const int v = warp >= 16, t = (tid - 384) & 127;
    constexpr int kPer = D / 16;  // chunks of 16 codes in a row
    const int row = t / kPer, k = t % kPer, sw = row & 7, c0 = 2 * (k & 3);
    const bool swap = k >= 4;
    const uint32_t at0 = uint32_t((c0 + (swap ? 1 : 0)) ^ sw) << 4, at1 = uint32_t((c0 + (swap ? 0 : 1)) ^ sw) << 4;
    unsigned char* dst = smem + (v ? C::kV : C::kK) + (k >> 2) * C::kHalfBytes + row * 128;
    const int empty = v ? kVEmpty : kKEmpty, full = v ? kVFull : kKFull;
    int slot = v, n = 0;
    uint32_t phase = 0;
    for (; it.valid(); it.next(p, sp, rg)) {
      for (int j = it.j0; j < it.j1; ++j, ++n) {
        (void)__all_sync(0xffffffffu, wait(st, kCodeFull + slot, phase));
        if (n > 0) (void)__all_sync(0xffffffffu, wait(st, empty, uint32_t(n - 1) & 1u));
        widen_tile<D>(smem + oCodes + slot * C::kCodeBytes + t * 16, dst, at0, at1, swap);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&st->bars[kCodeEmpty + slot]);
          mbar_arrive(&st->bars[full]);
        }
        slot += 2;
        if (slot >= slots) {
          slot -= slots;
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
    const int bs = p.block_size;
    // the token's table entry in tile j of `w` (-1: no position of the sequence), and its scales
    auto entry = [&](const Walk& w, int j) -> int {
      const int pos = w.q.base + j * kBN + t;
      return j < w.j1 && pos < w.q.e.L ? __ldg(p.block_tables + int64_t(w.s) * p.bt_stride + (pos >> sp.bs_shift)) : -1;
    };
    auto scales = [&](const Walk& w, int j, int e, float& ks, float& vs) {
      const int pos = w.q.base + j * kBN + t;
      ks = vs = 0.f;
      if (j < w.j1 && pos < w.q.e.L) {
        const int blk = e < 0 || int64_t(e) >= p.num_blocks ? 0 : e;  // (reported with the copies)
        const int64_t i = int64_t(blk) * p.ts_block + int64_t(w.kvh) * p.ts_head + (pos & (bs - 1));
        ks = __ldg(p.k_token_scales + i);
        vs = __ldg(p.v_token_scales + i);
      }
    };
    int item = 0, use = 0, step = 0;
    float ks = 0.f, vs = 0.f;
    int e1 = -1;
    if (it.valid()) {
      scales(it, it.j0, entry(it, it.j0), ks, vs);
      e1 = entry(it, it.j0 + 1);
    }
    while (it.valid()) {
      const ItemRows ir(p, sp, it);
      if (wg < ir.groups) {
        const Extent& e = it.q.e;
        const int nc = ir.half >> 4, ob = use & 1;
        const uint32_t tO = tmem + C::kO + ob * 128 + wg * 64 + lane_off;
        const float* qf = st->qf[item & 3][wg];
        unsigned char* ptile = smem + oP + wg * C::kPBytes;
        float vref = 0.f;
        Sums l;
#pragma unroll
        for (int i = 0; i < kHalfRows; ++i) l.a[i >> 4][i & 15] = 0.f;
        if (t < kHalfRows) {
          rw.m[t] = rw.limit[t] = -INFINITY;
          rw.shift[t] = 0.f;
        }
        group_sync(tk.id);
#pragma unroll 1
        for (int j = it.j0; j < it.j1; ++j, ++step) {
          float ks1, vs1;
          scales(it, j + 1, e1, ks1, vs1);
          e1 = entry(it, j + 2);
          const int pos = it.q.base + j * kBN + t;
          tk.ks = ks;
          tk.vs = vs;
          tk.valid = pos >= e.lo && pos < e.L;
          tk.cut = it.cut(j);
          tk.keep = ~0ull;
          if (tk.cut) {
            if (!tk.valid) {
              tk.keep = 0;
            } else if (p.tree_mask && pos >= e.P) {
              // the rows (node by node, g each) that see this node
              const int c = pos - e.P, r0 = wg * ir.half;
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
          (void)__all_sync(0xffffffffu, wait(st, kSFull + 2 * wg + (step & 1), uint32_t(step >> 1) & 1u));
          tc::fence_after();
          const uint32_t tS = tmem + C::kS + wg * 128 + (step & 1) * 64 + lane_off;
          const bool first = j == it.j0;
          softmax_step(st, rw, qf, tk, nc, tS, tO, ptile, kODone + wg, step, first, vref, l);
          fence_proxy_async_smem();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&st->bars[kPFull + wg]);
          ks = ks1;
          vs = vs1;
        }
        // the next item's first scales are on their way while this one's output is written
        Walk nx = it;
        nx.next(p, sp, rg);
        const int e0 = nx.valid() ? entry(nx, nx.j0) : -1;
        if (nx.valid()) e1 = entry(nx, nx.j0 + 1);
        (void)__all_sync(0xffffffffu, wait(st, kODone + wg, uint32_t(step - 1) & 1u));
        tc::fence_after();
        if (nx.valid()) scales(nx, nx.j0, e0, ks, vs);
        write_rows<D>(p, sp, it, ir, rw, tk.id, wg, q, lane, nc, tO, vref, l);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->bars[kOFree + 2 * wg + ob]);
        group_sync(tk.id);  // (the rows' state is this item's until all have written)
        ++use;
        it = nx;
      } else {
        it.next(p, sp, rg);
        if (it.valid()) {
          scales(it, it.j0, entry(it, it.j0), ks, vs);
          e1 = entry(it, it.j0 + 1);
        }
      }
      ++item;
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
  return p.head_dim == 128 ? launch_tree_i8_tpl<128>(p, sp, stream) : launch_tree_i8_tpl<64>(p, sp, stream);
}

}  // namespace pkv
