// decode_e2m1.cu — decode attention of few query heads a KV head (at most 16) over a 4-bit cache.
//
// For a sequence's row h, position j, codes ck, cv and group scales gk, gv (a column's group is its
// 16), and the caches' factors fk, fv of the KV head:
//   z_j = (q . (ck_j gk_j)) fk scale log2 e,  p_j = 2^(z_j - m),
//   out = fv sum_j p_j (cv_j gv_j) / sum_j p_j        with any m; here the largest z_j so far.
//
// What bounds it is HBM: 2 (D / 2 + D / 16) bytes a position and KV head, and close behind the
// instructions that widen 2 D codes: at the memory's rate an SM has about four issue slots a
// position and KV head for each of its lanes' eight codes.  So a code is widened once, in registers:
// a pair of codes is one conversion to f16 and one product with the group's scale, both exact (see
// e2m1_codes.cuh), and the result is an operand of the small transposed products (mma m16n8k16,
// tokens or columns x heads), in the order that the loads bring it (a permutation of the columns
// that the queries share).  A lane's 16 or 32 codes of a K row lie in one or two groups, its D / 8
// codes of a V row in one; V's pairs are two tokens' codes of a column, brought together by two
// shifts and two selections for sixteen codes, and their scales by a transposition of 8 tokens x 8
// groups (movmatrix).
//
// A warp takes 32 positions of a tile of 128 and brings them itself, two steps ahead, into a ring
// of three in shared memory (asynchronous copies of 16 bytes a lane).  A warp has its own reference
// m of a row (moved when a token exceeds it by 2^8) and its own sums; the four are folded at an
// item's end, in order.  Weights are rounded to f16, half a step, 2^-11, down to 2^-21 of the row's
// largest, 2^-32 of that below.  Everything else is exact or binary32.
//
// 8 sequences of 32768 positions, 32 : 8 heads of 128 (302 MB): 65 us, 4.6 TB/s, 36 M warp
// instructions; the copies alone take 54 us, the instructions alone 57.  64 sequences of 129 to 2048
// positions (82 MB): 29 us, of it about 2 for the work split, 4 to the first codes and 6 for the fold
// of split rows.  Tried without gain: four stages, two or four blocks an SM (82 and 70 us for the long
// sequences, three 65), scores and products of two halves interleaved, table entries two steps
// ahead, sums by products with ones, the next item begun before the fold, the fold by the block
// that finishes last.
#include <algorithm>
#include <mutex>

#include "decode_few.cuh"
#include "e2m1_codes.cuh"

namespace pkv {
namespace decode_e2m1 {

using namespace decode_few;
using tree::kBN;
using tree::kGap;
using tree::Range;
using tree::Walk;

constexpr int kStages = 3;  // of a warp's ring
constexpr int blocks_per_sm(int nt) { return nt == 1 ? 3 : 2; }
// A row's weights are 2^(z - m + kTop): at most 2^15 with a reference that lags by 2^kGap.
constexpr float kTop = 7.f;
constexpr float kNoLift = 3.402823466e38f;  // kTop - m before the first score, with which every score moves m

__device__ __forceinline__ uint32_t mul_pair(uint32_t a, __half2 s) {
  const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&a), s);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }

__device__ __forceinline__ void copy16(uint32_t dst, const unsigned char* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const unsigned char* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void end_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void load_shared(uint32_t a, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
}
__device__ __forceinline__ void load_shared(uint32_t a, uint32_t (&w)[2]) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
}
__device__ __forceinline__ void load_shared(uint32_t a, uint32_t (&w)[1]) {
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(a));
}
// Two group scales (one, at D = 64), as they are stored.
template <int D>
__device__ __forceinline__ uint32_t load_scales(uint32_t a) {
  uint32_t x;
  if (D == 128) asm volatile("ld.shared.u16 %0, [%1];" : "=r"(x) : "r"(a));
  else asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(a));
  return x;
}

// A stage of the ring: 32 positions' rows of K, of V, and the group scales of both.
//
// Eight rows lie in 8 kRow bytes.  Lane (g, t) reads 16 (D = 64: 8) bytes of row g of K and 8 (4) of
// rows 2t and 2t + 1 of V; where a row goes, and its halves, makes neither meet a bank twice.
template <int D>
struct Stage {
  static constexpr int kRow = D / 2, kGroups = D / 16;  // bytes and groups of a row
  static constexpr uint32_t kV = 32 * kRow, kKScales = 64 * kRow, kVScales = kKScales + 32 * kGroups;
  static constexpr uint32_t kBytes = kVScales + 32 * kGroups;
  __device__ static __forceinline__ uint32_t at(int r, int byte) {
    if (D == 128) return (r ^ ((r >> 1) & 1)) * kRow + (byte ^ ((r & 4) << 3));  // (the upper rows' halves swapped)
    return ((r & 4) | ((r >> 1) & 1) | (((r ^ (r >> 2)) & 1) << 1)) * kRow + byte;
  }
};
template <int D, int NT>
constexpr size_t smem_bytes() {
  static_assert(sizeof(Rows<D, NT>) <= kWarps * kStages * Stage<D>::kBytes, "the rows take the rings' place");
  return size_t(kWarps) * kStages * Stage<D>::kBytes;
}

// NT x 8 rows: the query heads of a KV head.  Blocks of 2^kShift tokens, 8 to 32.
template <int D, int NT, int kShift>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(NT))
decode_e2m1_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeSplit sp) {
  using S = Stage<D>;
  constexpr int kRow = S::kRow, kGroups = S::kGroups, kMask = (1 << kShift) - 1;
  constexpr int kK = D / 32, kV = D / 64;  // words of a row of K and of V that a lane holds
  extern __shared__ __align__(128) unsigned char smem[];  // the rings; at an item's end the warps' O
  __shared__ Shared<D, NT> sh;
  Rows<D, NT>& rows = *reinterpret_cast<Rows<D, NT>*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing of the caller's is read before
  asm volatile("griddepcontrol.launch_dependents;");
  (void)tree::find_range<kThreads>(p, sp, &sh.range, sh.warp_sum, 0);
  const Range* rg = &sh.range;
  Walk it;
  it.start(p, sp, rg);
  int64_t at = rg->from;
  TreeSplit::Tail tail = {0, 0, 0, 0};
  const uint32_t ring = smem_addr(smem) + warp * kStages * S::kBytes;
  // a copy of codes: of row crow of eight rows, 16 bytes from cbyte on (at D = 64 of 2 x 8 rows)
  const int crow = D == 128 ? lane >> 2 : (lane >> 1) & 7, cbyte = (D == 128 ? lane & 3 : lane & 1) * 16;
  const int ceight = D == 128 ? 0 : 8 * (lane >> 4);
  const uint32_t block_bytes = uint32_t(p.cs_block), block_scales = uint32_t(p.ts_block);
  const uint32_t cto = ring + S::at(crow, cbyte) + ceight * kRow;
  const uint32_t kfrom = ring + S::at(g, 4 * kK * t);
  const uint32_t vfrom0 = ring + S::kV + S::at(2 * t, 4 * kV * g), vfrom1 = ring + S::kV + S::at(2 * t + 1, 4 * kV * g);
  const uint32_t gfrom = ring + S::kKScales + g * kGroups + (D / 64) * t;  // of token g, the lane's groups of K
  for (; it.valid(); it.next(p, sp, rg)) {
    const int64_t head = int64_t(it.kvh) * p.cs_head + (crow + (ceight & kMask)) * kRow + cbyte;
    const unsigned char* kc = static_cast<const unsigned char*>(p.key_cache) + head;
    const unsigned char* vc = static_cast<const unsigned char*>(p.value_cache) + head;
    // the warp's steps: its 32 positions of each tile that start inside the context
    const int L = it.q.e.L, lo = it.q.e.lo, first = it.q.base + it.j0 * kBN + 32 * warp;
    const int steps = min(it.j1 - it.j0, (L - first + kBN - 1) / kBN);
    // The table's entries of the lane's positions, a step's each time.  (0 where there is none:
    // positions behind the context are read from block 0, whose numbers have no part: their scores
    // are hidden, their value scales zero.)
    int entry_pos = first + lane;
    const int32_t* entry_at = p.block_tables + int64_t(it.s) * p.bt_stride + (entry_pos >> kShift);
    auto entry = [&]() -> uint32_t {
      uint32_t e = 0;
      if (entry_pos < L) {
        e = uint32_t(__ldg(entry_at));
        if (e >= uint32_t(p.num_blocks)) {
          raise_device_error(p.err, kErrTableEntry);
          e = 0;
        }
      }
      entry_pos += kBN;
      entry_at += kBN >> kShift;
      return e;
    };
    // A step's first position is a block's first, so eight positions from a multiple of 8 on share a
    // block and lie at known places in it.
    constexpr int kPer = 16 / kGroups, kLanes = 32 / kPer;  // tokens' scales of 16 bytes, lanes for a tensor's
    const bool of_v = lane >= kLanes;
    const int stok = lane % kLanes * kPer;
    const unsigned char* sc = (of_v ? p.v_group_scales : p.k_group_scales) + int64_t(it.kvh) * p.ts_head + (stok & kMask) * kGroups;
    const uint32_t sto = ring + (of_v ? S::kVScales : S::kKScales) + stok * kGroups;
    auto copy_stage = [&](uint32_t e, uint32_t off) {
      constexpr int kTokens = D == 128 ? 8 : 16;  // of a copy
      const unsigned char *k = kc, *v = vc;
#pragma unroll
      for (int c = 0; c < 32; c += kTokens) {
        if ((c & kMask) == 0 || kTokens > kMask) {  // (another block)
          const uint64_t src = uint64_t(__shfl_sync(0xffffffffu, e, c + (kTokens > kMask ? ceight : 0))) * block_bytes;
          k = kc + src;
          v = vc + src;
        }
        copy16(cto + off + c * kRow, k + (c & kMask) * kRow);
        copy16(cto + off + c * kRow + S::kV, v + (c & kMask) * kRow);
      }
      if (sp.vec_scales) {
        const uint64_t src = uint64_t(__shfl_sync(0xffffffffu, e, stok)) * block_scales;
        if (lane < 2 * kLanes) copy16(sto + off, sc + src);
      } else {  // (words of four, at any multiple of them)
#pragma unroll 1
        for (int c = 0; c < kGroups / 2; ++c) {  // 32 kGroups / 4 words a tensor, K's first
          const bool v = c >= kGroups / 4;
          const int byte = 4 * (32 * (c - (v ? kGroups / 4 : 0)) + lane), tok = byte / kGroups;
          const int64_t src = int64_t(it.kvh) * p.ts_head + uint64_t(__shfl_sync(0xffffffffu, e, tok)) * block_scales +
                              (tok & kMask) * kGroups + byte % kGroups;
          copy4(ring + off + (v ? S::kVScales : S::kKScales) + byte, (v ? p.v_group_scales : p.k_group_scales) + src);
        }
      }
    };
    uint32_t e_next = entry();
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) {
      const uint32_t e = e_next;
      e_next = entry();
      if (j < steps) copy_stage(e, j * S::kBytes);
      end_copies();
    }

    // the queries: B of the scores' product, columns permuted as K's are
    uint32_t qb[NT][4 * kK];
    float qf[NT][2];  // score factors of rows 2t, 2t + 1
    const float fk = p.qk_scale_log2 * (p.k_head_scales ? __ldg(p.k_head_scales + it.kvh) : 1.f);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint4 x[kK];
#pragma unroll
      for (int c = 0; c < kK; ++c) {
        x[c] = make_uint4(0u, 0u, 0u, 0u);
        if (8 * n + g < p.group)
          x[c] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.query) + it.q.e.q0 * p.q_stride_t +
                                                 int64_t(it.kvh * p.group + 8 * n + g) * p.q_stride_h + 8 * (kK * t + c));
      }
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < kK; ++c) {
        float f[8];
        Chunk<BF16>::expand(x[c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int shift = i8::query_shift(top);
      const float s = i8::power(shift), f = fk * i8::power(-shift);
#pragma unroll
      for (int c = 0; c < kK; ++c) {
        float y[8];
        Chunk<BF16>::expand(x[c], y);
#pragma unroll
        for (int i = 0; i < 4; ++i) qb[n][4 * c + i] = half2_bits(y[2 * i] * s, y[2 * i + 1] * s);
      }
      qf[n][0] = __shfl_sync(0xffffffffu, f, 8 * t);
      qf[n][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }

    float m[NT][2], lift[NT][2], l[NT][2];  // of rows 2t, 2t + 1: m, kTop - m, sum over this lane's tokens
    float o[NT][4 * kV][4];                 // O^T: see the products
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      lift[n][0] = lift[n][1] = kNoLift;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * kV; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }

    uint32_t off = 0, off_next = (kStages - 1) * S::kBytes;  // this step's stage, and the one that is filled
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
      const int pos0 = first + j * kBN;
      wait_copies<kStages - 2>();
      __syncwarp();  // every lane's copies have landed, and every lane has read the stage before
      if (j + kStages - 1 < steps) copy_stage(e_next, off_next);
      end_copies();
      e_next = entry();
      off_next = off;
      // S^T: tokens 16 u + g, + 8; rows 2t, 2t + 1
      float s[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t x[2][kK];
        __half2 gs[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          load_shared(kfrom + off + (2 * u + h) * 8 * kRow, x[h]);
          gs[h] = as_half2(e2m1::scales2(load_scales<D>(gfrom + off + (2 * u + h) * 8 * kGroups)));
        }
#pragma unroll
        for (int c = 0; c < kK; ++c) {
          // (a word is half a group: of the lane's first or, from word 2 on, its second)
          const __half2 sa = c < 2 ? __low2half2(gs[0]) : __high2half2(gs[0]);
          const __half2 sb = c < 2 ? __low2half2(gs[1]) : __high2half2(gs[1]);
          uint32_t a[4], b[4];
          e2m1::widen8(x[0][c], a);
          e2m1::widen8(x[1][c], b);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = mul_pair(a[i], sa);
            b[i] = mul_pair(b[i], sb);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (c == 0) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.f;
            mma(s[u][n], a[0], b[0], a[1], b[1], qb[n][4 * c], qb[n][4 * c + 1]);
            mma(s[u][n], a[2], b[2], a[3], b[3], qb[n][4 * c + 2], qb[n][4 * c + 3]);
          }
        }
      }
      // the weights' exponents
      float z[2][NT][4];
      const bool cut = pos0 + 32 > L || pos0 < lo;  // some token is not attended to
      auto exponents = [&]() {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[u][n][i] = fmaf(s[u][n][i], qf[n][i & 1], lift[n][i & 1]);
        if (cut) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int a = pos0 + 16 * u + 8 * h + g;
              if (a >= L || a < lo) {
#pragma unroll
                for (int n = 0; n < NT; ++n) z[u][n][2 * h] = z[u][n][2 * h + 1] = -INFINITY;
              }
            }
        }
      };
      exponents();
      float over = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) over = fmaxf(over, z[u][n][i]);
      if (__any_sync(0xffffffffu, over > kGap + kTop)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float a[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float mx = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int tok = pos0 + 16 * u + 8 * h + g;
                const float x = s[u][n][2 * h + r] * qf[n][r];
                mx = fmaxf(mx, cut && (tok >= L || tok < lo) ? -INFINITY : x);
              }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const bool go = mx > m[n][r] + kGap || (m[n][r] == -INFINITY && mx > -INFINITY);
            a[r] = go ? fast_exp2(m[n][r] - mx) : 1.f;  // (0 from -infinity)
            if (go) {
              m[n][r] = mx;
              lift[n][r] = kTop - mx;
            }
            l[n][r] *= a[r];
          }
#pragma unroll
          for (int i = 0; i < 4 * kV; ++i) {
            o[n][i][0] *= a[0];
            o[n][i][1] *= a[1];
            o[n][i][2] *= a[0];
            o[n][i][3] *= a[1];
          }
        }
        exponents();
      }
      // the weights, as B of the products
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float x = fast_exp2(z[u][n][2 * h]), y = fast_exp2(z[u][n][2 * h + 1]);
            l[n][0] += x;
            l[n][1] += y;
            pb[u][n][h] = transpose8x8(half2_bits(x, y));
          }
      // O^T: four products for each of the lane's words of V; the first 8 rows of product i are the
      // lanes' columns 2 i of the word, the others the columns after them
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t v[2][2][kV];  // rows 2t, 2t + 1, 8 rows further: D / 8 codes from D / 8 g on
        __half2 gs[2];         // the lane's group's scales of the two rows
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          load_shared(vfrom0 + off + (2 * u + h) * 8 * kRow, v[h][0]);
          load_shared(vfrom1 + off + (2 * u + h) * 8 * kRow, v[h][1]);
          uint32_t two = e2m1::scales2(
              load_scales<D>(gfrom + off + (S::kVScales - S::kKScales) + (2 * u + h) * 8 * kGroups));
          if (D == 64) two = __byte_perm(two, two, 0x1010);  // (each group twice: two lanes' columns)
          two = transpose8x8(two);
          if (cut) {
            const int a = pos0 + 16 * u + 8 * h + 2 * t;
            if (a >= L || a < lo) two &= 0xffff0000u;
            if (a + 1 >= L || a + 1 < lo) two &= 0xffffu;
          }
          gs[h] = as_half2(two);
        }
#pragma unroll
        for (int w = 0; w < kV; ++w) {
          uint32_t even[2][4], odd[2][4];  // a column of two tokens, side by side
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = v[h][0][w], y = v[h][1][w];
            e2m1::widen8((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), even[h]);
            e2m1::widen8(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), odd[h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              even[h][i] = mul_pair(even[h][i], gs[h]);
              odd[h][i] = mul_pair(odd[h][i], gs[h]);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma(o[n][4 * w + i], even[0][i], odd[0][i], even[1][i], odd[1][i], pb[u][n][0], pb[u][n][1]);
        }
      }
      off = off + S::kBytes == kStages * S::kBytes ? 0 : off + S::kBytes;
    }

    // the warps' results together
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], x);
        if (g == 0) {
          sh.m[warp][8 * n + 2 * t + r] = m[n][r];
          sh.l[warp][8 * n + 2 * t + r] = l[n][r];
        }
#pragma unroll
        for (int w = 0; w < 2 * kV; ++w)
          *reinterpret_cast<float4*>(&rows.o[warp][8 * n + 2 * t + r][8 * kV * g + 4 * w]) =
              make_float4(o[n][2 * w][r], o[n][2 * w][2 + r], o[n][2 * w + 1][r], o[n][2 * w + 1][2 + r]);
      }
    }
    __syncthreads();
    fold_warps<D, NT>(p, sp, it, sh, rows, p.v_head_scales ? __ldg(p.v_head_scales + it.kvh) : p.v_scale);
    __syncthreads();  // (the rings are free again)
    if (it.begins() && !it.ends()) {
      tail.row0 = it.q.e.q0;
      tail.nodes = 1;
      tail.kvh = it.kvh;
      tail.last = int((at - it.u0 + it.q.tiles + rg->cost - 1) / rg->share);
    }
    at += it.u1 - it.u0;
  }
  if (tid == 0) sp.tails[blockIdx.x] = tail;
}

}  // namespace decode_e2m1

namespace {

template <int D, int NT, int kShift>
cudaError_t launch_shift(const TreeParams& p, const TreeSplit& sp, cudaStream_t stream) {
  constexpr size_t kSmem = decode_e2m1::smem_bytes<D, NT>();
  static_assert(decode_e2m1::blocks_per_sm(NT) * (kSmem + sizeof(decode_few::Shared<D, NT>) + 1024) <= 228 * 1024,
                "shared memory");
  constexpr int kDevices = 64;
  auto kern = decode_e2m1::decode_e2m1_kernel<D, NT, kShift>;
  static std::once_flag once[kDevices];
  static cudaError_t set[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    set[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
  });
  if (set[dev] != cudaSuccess) return set[dev];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sp.grid));
  cfg.blockDim = dim3(decode_few::kThreads);
  cfg.dynamicSmemBytes = kSmem;
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

template <int D, int NT>
cudaError_t launch_decode_e2m1_tpl(const TreeParams& p, const TreeSplit& sp, cudaStream_t stream) {
  if (p.block_size == 8) return launch_shift<D, NT, 3>(p, sp, stream);
  return p.block_size == 16 ? launch_shift<D, NT, 4>(p, sp, stream) : launch_shift<D, NT, 5>(p, sp, stream);
}

}  // namespace

// At most 16 heads: 8 sequences of 32768 positions take 65, 66 and 88 us with 4, 8 and 16 heads a KV
// head here, 132 us in the tree kernel (tree_e2m1.cu) whatever their number; 64 sequences of 129 to
// 2048 positions 29, 31 and 41 us, 69 to 77 there.  Blocks of 2 and 4 tokens do not hold eight
// positions in a row.
bool decode_e2m1_supported(const TreeParams& p) {
  if (p.q_dtype != kBF16 || p.kv_dtype != kE2M1 || p.query_start_loc || p.group > 16 || p.block_size < 8) return false;
  if ((p.cs_block | p.ts_block) >> 32 || p.num_blocks > 0x7fffffff) return false;  // (multiplied in 32 bits)
  return (reinterpret_cast<uintptr_t>(p.query) & 15) == 0 && (p.q_stride_t & 7) == 0 && (p.q_stride_h & 7) == 0;
}

int decode_e2m1_blocks_per_sm(int group) { return decode_e2m1::blocks_per_sm(group <= 8 ? 1 : 2); }

cudaError_t launch_decode_e2m1(const TreeParams& p, TreeSplit sp, cudaStream_t stream) {
  sp.item_nodes = sp.tq = 1;
  sp.vec_scales = !((reinterpret_cast<uintptr_t>(p.k_group_scales) | reinterpret_cast<uintptr_t>(p.v_group_scales) |
                     p.ts_block | p.ts_head) & 15);
  if (p.head_dim == 128)
    return p.group <= 8 ? launch_decode_e2m1_tpl<128, 1>(p, sp, stream) : launch_decode_e2m1_tpl<128, 2>(p, sp, stream);
  return p.group <= 8 ? launch_decode_e2m1_tpl<64, 1>(p, sp, stream) : launch_decode_e2m1_tpl<64, 2>(p, sp, stream);
}

}  // namespace pkv
