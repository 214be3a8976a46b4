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
// A warp takes 32 positions of a tile of 128, its loads of K a step ahead and of V during the
// scores.  A warp has its own reference m of a row (moved when a token exceeds it by 2^8) and its
// own sums; the four are folded at an item's end, in order.  Weights are rounded to f16, half a
// step, 2^-11, down to 2^-21 of the row's largest, 2^-32 of that below.  Everything else is exact or
// binary32.
#include "decode_few.cuh"
#include "e2m1_codes.cuh"

namespace pkv {
namespace decode_e2m1 {

using namespace decode_few;
using tree::kBN;
using tree::kGap;
using tree::Range;
using tree::Walk;

// A row's weights are 2^(z - m + kTop): under 2^15 with a reference that lags by 2^kGap.
constexpr float kTop = 7.f;

__device__ __forceinline__ uint32_t mul_pair(uint32_t a, __half2 s) {
  const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&a), s);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }

// 16 bytes of a head of 128 columns' row, 8 of one of 64
template <int D>
__device__ __forceinline__ void load_codes(const unsigned char* p, uint32_t (&w)[D / 32]) { load_words(p, w); }
__device__ __forceinline__ void load_word(const unsigned char* p, uint32_t (&w)[2]) { load_words(p, w); }
__device__ __forceinline__ void load_word(const unsigned char* p, uint32_t (&w)[1]) {
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
}
// The group scales of lane (g, t)'s token: groups 2t, 2t + 1 of 8, or group t of 4.
template <int D>
__device__ __forceinline__ uint32_t load_scales(const unsigned char* p) {
  return D == 128 ? uint32_t(*reinterpret_cast<const uint16_t*>(p)) : uint32_t(*p);
}

// NT x 8 rows: the query heads of a KV head.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
decode_e2m1_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeSplit sp) {
  constexpr int kRow = D / 2, kGroups = D / 16;  // bytes and groups of a row
  constexpr int kK = D / 32;                     // words of a K row that a lane holds
  constexpr int kV = D / 64;                     // and of a V row
  __shared__ Shared<D, NT> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing of the caller's is read before
  asm volatile("griddepcontrol.launch_dependents;");
  (void)tree::find_range<kThreads>(p, sp, &sh.range, sh.warp_sum, 0);
  const Range* rg = &sh.range;
  Walk it;
  it.start(p, sp, rg);
  const int bs_mask = p.block_size - 1;
  int64_t at = rg->from;
  TreeSplit::Tail tail = {0, 0, 0, 0};
  for (; it.valid(); it.next(p, sp, rg)) {
    const int32_t* table = p.block_tables + int64_t(it.s) * p.bt_stride;
    const int64_t head = int64_t(it.kvh) * p.cs_head, ghead = int64_t(it.kvh) * p.ts_head;
    // the lane's part of token g's row of K (of tokens 2t, 2t + 1 of V), and of token g's scales
    const unsigned char* kc = static_cast<const unsigned char*>(p.key_cache) + head + g * kRow + 4 * kK * t;
    const unsigned char* vc = static_cast<const unsigned char*>(p.value_cache) + head + 2 * t * kRow + 4 * kV * g;
    const unsigned char* kg = p.k_group_scales + ghead + g * kGroups + (D / 64) * t;
    const unsigned char* vg = p.v_group_scales + ghead + g * kGroups + (D / 64) * t;
    const int L = it.q.e.L, lo = it.q.e.lo, steps = it.j1 - it.j0;
    int pos = it.q.base + it.j0 * kBN + 32 * warp + lane;
    auto entry = [&](int at) -> int {
      if (at >= L) return 0;
      int e = __ldg(table + (at >> sp.bs_shift));
      if (e < 0 || int64_t(e) >= p.num_blocks) {
        raise_device_error(p.err, kErrTableEntry);
        e = 0;
      }
      return e;
    };
    // Eight positions from a multiple of 8 on share a block (of at least 8): its entry comes from the
    // first one's lane.  (Positions past the context are read from block 0, whose numbers have no
    // part: their scores are hidden, their value scales zero.)
    int blk[2][2];
    uint32_t kreg[2][2][kK];  // K rows g, g + 8 of 16 tokens
    uint32_t ks[2][2], vs[2][2];  // their group scales, as they are stored
    auto load_k = [&](int e) {
      const int first = pos - lane;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          blk[u][h] = __shfl_sync(0xffffffffu, e, 16 * u + 8 * h);
          const int in = (first + 16 * u + 8 * h) & bs_mask;
          load_codes<D>(kc + int64_t(blk[u][h]) * p.cs_block + in * kRow, kreg[u][h]);
          const int64_t sc = int64_t(blk[u][h]) * p.ts_block + in * kGroups;
          ks[u][h] = load_scales<D>(kg + sc);
          vs[u][h] = load_scales<D>(vg + sc);
        }
    };
    load_k(entry(pos));
    int e_next = steps > 1 ? entry(pos + kBN) : 0;

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

    float m[NT][2], l[NT][2];  // of rows 2t, 2t + 1 (l: this lane's tokens)
    float o[NT][4 * kV][4];    // O^T: see the products
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * kV; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }

#pragma unroll 1
    for (int j = 0; j < steps; ++j, pos += kBN) {
      const int pos0 = pos - lane;
      if (pos0 >= L) break;  // (the last tile: nothing for this warp)
      // V rows 2t, 2t + 1, 2t + 8, 2t + 9 of 16 tokens, D / 8 codes from D / 8 g on
      uint32_t v[2][4][kV];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const unsigned char* src =
              vc + int64_t(blk[u][h]) * p.cs_block + ((pos0 + 16 * u + 8 * h) & bs_mask) * kRow;
          load_word(src, v[u][2 * h]);
          load_word(src + kRow, v[u][2 * h + 1]);
        }
      // S^T: tokens 16 u + g, + 8; rows 2t, 2t + 1
      float s[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.f;
        const __half2 ga = as_half2(e2m1::scales2(ks[u][0])), gb = as_half2(e2m1::scales2(ks[u][1]));
#pragma unroll
        for (int c = 0; c < kK; ++c) {
          // (a word is half a group: of the lane's first or, at D = 128, from word 2 on its second)
          const __half2 sa = c < 2 ? __low2half2(ga) : __high2half2(ga), sb = c < 2 ? __low2half2(gb) : __high2half2(gb);
          uint32_t a[4], b[4];
          e2m1::widen8(kreg[u][0][c], a);
          e2m1::widen8(kreg[u][1][c], b);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = mul_pair(a[i], sa);
            b[i] = mul_pair(b[i], sb);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma(s[u][n], a[0], b[0], a[1], b[1], qb[n][4 * c], qb[n][4 * c + 1]);
            mma(s[u][n], a[2], b[2], a[3], b[3], qb[n][4 * c + 2], qb[n][4 * c + 3]);
          }
        }
      }
      // the value scales of the lane's group for tokens 16 u + 8 h + 2t, + 1
      __half2 gv[2][2];
      const bool cut = pos0 + 32 > L || pos0 < lo;  // some token is not attended to
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t two = e2m1::scales2(vs[u][h]);
          if (D == 64) two = __byte_perm(two, two, 0x1010);  // (each group twice: eight columns a lane)
          two = transpose8x8(two);
          if (cut) {
            const int a = pos0 + 16 * u + 8 * h + 2 * t;
            if (a >= L || a < lo) two &= 0xffff0000u;
            if (a + 1 >= L || a + 1 < lo) two &= 0xffffu;
          }
          gv[u][h] = as_half2(two);
        }
      // the next step's codes and scales, and the entries of the one after it
      pos += kBN;
      if (j + 1 < steps) {
        load_k(e_next);
        e_next = j + 2 < steps ? entry(pos + kBN) : 0;
      }
      pos -= kBN;
      bool move = false;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at_tok = pos0 + 16 * u + 8 * h + g;
          const bool hidden = cut && (at_tok >= L || at_tok < lo);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& z = s[u][n][2 * h + r];
              z = hidden ? -INFINITY : z * qf[n][r];
              move |= z > m[n][r] + kGap;
            }
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float a[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float mx = fmaxf(fmaxf(s[0][n][r], s[0][n][2 + r]), fmaxf(s[1][n][r], s[1][n][2 + r]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const bool go = mx > m[n][r] + kGap || (m[n][r] == -INFINITY && mx > -INFINITY);
            a[r] = go ? fast_exp2(m[n][r] - mx) : 1.f;  // (0 from -infinity)
            if (go) m[n][r] = mx;
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
      }
      // the weights, as B of the products
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float r0 = m[n][0] == -INFINITY ? 0.f : m[n][0] - kTop;
        const float r1 = m[n][1] == -INFINITY ? 0.f : m[n][1] - kTop;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float x = fast_exp2(s[u][n][2 * h] - r0), y = fast_exp2(s[u][n][2 * h + 1] - r1);
            l[n][0] += x;
            l[n][1] += y;
            pb[u][n][h] = transpose8x8(half2_bits(x, y));
          }
      }
      // O^T: four products for each of the lane's words of V; the first 8 rows of product i are the
      // lanes' columns 2 i of the word, the others the columns after them
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int w = 0; w < kV; ++w) {
          uint32_t even[2][4], odd[2][4];  // a column of two tokens, side by side
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = v[u][2 * h][w], y = v[u][2 * h + 1][w];
            e2m1::widen8((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), even[h]);
            e2m1::widen8(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), odd[h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              even[h][i] = mul_pair(even[h][i], gv[u][h]);
              odd[h][i] = mul_pair(odd[h][i], gv[u][h]);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma(o[n][4 * w + i], even[0][i], odd[0][i], even[1][i], odd[1][i], pb[u][n][0], pb[u][n][1]);
        }
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
          *reinterpret_cast<float4*>(&sh.o[warp][8 * n + 2 * t + r][8 * kV * g + 4 * w]) =
              make_float4(o[n][2 * w][r], o[n][2 * w][2 + r], o[n][2 * w + 1][r], o[n][2 * w + 1][2 + r]);
      }
    }
    __syncthreads();
    fold_warps<D, NT>(p, sp, it, sh, p.v_head_scales ? __ldg(p.v_head_scales + it.kvh) : p.v_scale);
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

template <int D, int NT>
cudaError_t launch_decode_e2m1_tpl(const TreeParams& p, const TreeSplit& sp, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sp.grid));
  cfg.blockDim = dim3(decode_few::kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, decode_e2m1::decode_e2m1_kernel<D, NT>, p, sp);
  note_launch();
  if (e != cudaSuccess) return e;
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_tree_merge(p, sp, stream);
}

}  // namespace

// Blocks of 2 and 4 tokens do not hold eight positions in a row.
bool decode_e2m1_supported(const TreeParams& p) {
  if (p.q_dtype != kBF16 || p.kv_dtype != kE2M1 || p.query_start_loc || p.group > 16 || p.block_size < 8) return false;
  return (reinterpret_cast<uintptr_t>(p.query) & 15) == 0 && (p.q_stride_t & 7) == 0 && (p.q_stride_h & 7) == 0;
}

int decode_e2m1_blocks_per_sm(int group) { return group <= 8 ? 3 : 2; }

cudaError_t launch_decode_e2m1(const TreeParams& p, TreeSplit sp, cudaStream_t stream) {
  sp.item_nodes = sp.tq = 1;
  if (p.head_dim == 128)
    return p.group <= 8 ? launch_decode_e2m1_tpl<128, 1>(p, sp, stream) : launch_decode_e2m1_tpl<128, 2>(p, sp, stream);
  return p.group <= 8 ? launch_decode_e2m1_tpl<64, 1>(p, sp, stream) : launch_decode_e2m1_tpl<64, 2>(p, sp, stream);
}

}  // namespace pkv
