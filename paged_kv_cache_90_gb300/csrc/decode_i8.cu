// decode_i8.cu — decode attention of few query heads a KV head (at most 16) over a
// token-scaled int8 cache.
//
// For a sequence's row h, position j and the caches' codes ck, cv with scales sk, sv:
//   z_j = sk_j (q . ck_j) scale log2 e,  p_j = 2^(z_j - m),  out = sum_j (p_j sv_j) cv_j / sum_j p_j
// with any m; here the largest z_j + log2 sv_j (i8::scale_exponent), which puts the row's largest
// product p_j sv_j near the top of f16.
//
// What bounds it is HBM: 2 (D + 4) bytes a position and KV head, for 8 heads of 128 about 31
// operations a byte.  What it must not do is spend instructions: a code is widened once, in
// registers, and goes from its load straight into a tensor-core operand.  So the products are
// the small transposed ones (mma m16n8k16, tokens or columns x heads): their A operand is 16
// tokens of K in the order that the loads bring them (a permutation of the columns that the
// queries share), or V^T from pairs of tokens' bytes, and O^T stays in 32 accumulators a lane.
// The fifth-generation MMAs take operands from shared memory only: there the same codes are
// copied, widened, written back and waited for by four roles, 33 M warp instructions a launch
// for 64 sequences of 1100 positions and 83 us at best; here 38 us (4.0 TB/s), and 97 us (5.7 TB/s)
// for 8 of 32768.
//
// A warp takes 32 positions of a tile of 128, its loads of K a step ahead and of V during the
// scores; 12 warps on an SM keep about 90 KB on the way.  A warp has its own reference m of a row
// (moved when a token exceeds it by 2^8) and its own sums; the four are folded at an item's end,
// in order.  The products p_j sv_j are rounded to f16: half a step, 2^-11, down to 2^-20 of the
// row's largest, 2^-31 of that below.  Everything else is exact (the widening) or binary32.
#include "i8_codes.cuh"
#include "tree_split.cuh"

namespace pkv {
namespace decode_i8 {

using tree::kBN;
using tree::kGap;
using tree::Range;
using tree::Walk;

constexpr int kWarps = 4, kThreads = 32 * kWarps;

__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[4]) {
  const uint4 v = load16(p);
  w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
}
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[2]) {
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
}

// f16 x f16 -> f32, 16 x 8 += 16 x 16 times 16 x 8.  Lane (g, t) = (lane / 4, lane % 4): a0 is
// A[g][2t, 2t+1], a1 A[g+8][..], a2 and a3 the same 8 columns further; b0 is B[2t, 2t+1][g], b1 8
// rows further; c is C[g][2t], C[g][2t+1], C[g+8][2t], C[g+8][2t+1].
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int NT>
struct Shared {
  Range range;
  longlong2 warp_sum[kWarps];
  float m[kWarps][8 * NT], l[kWarps][8 * NT];
  alignas(16) float o[kWarps][8 * NT][D + 4];
};

// NT x 8 rows: the query heads of a KV head.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
decode_i8_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ TreeSplit sp) {
  constexpr int kC = D / 64;    // 64-column halves of a row
  constexpr int kW = D / 32;    // words of a V row that a lane holds
  constexpr int kRows = 8 * NT;
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
    const int64_t head = int64_t(it.kvh) * p.cs_head, thead = int64_t(it.kvh) * p.ts_head;
    const unsigned char* kc = static_cast<const unsigned char*>(p.key_cache) + head;
    const unsigned char* vc = static_cast<const unsigned char*>(p.value_cache) + head;
    const int L = it.q.e.L, lo = it.q.e.lo, steps = it.j1 - it.j0;
    // the lane's token of the step looked up last, and of the one before it
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
    float ks = 0.f, vs = 0.f;
    int64_t row = 0;         // the lane's token's row in the caches (a valid one where it has none)
    uint4 kreg[2][2][kC];    // K rows g, g + 8 of 16 tokens: 16 codes from 16 t on, of each half
    auto load_k = [&](int e) {
      const bool there = pos < L;
      row = there ? int64_t(e) * p.cs_block + int64_t((pos & bs_mask) * D) : 0;
      const int64_t sc = there ? int64_t(e) * p.ts_block + thead + (pos & bs_mask) : 0;
      ks = there ? __ldg(p.k_token_scales + sc) : 0.f;
      vs = there ? __ldg(p.v_token_scales + sc) : 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const unsigned char* src = kc + __shfl_sync(0xffffffffu, row, 16 * u + 8 * h + g) + 16 * t;
#pragma unroll
          for (int c = 0; c < kC; ++c) kreg[u][h][c] = load16(src + 64 * c);
        }
    };
    load_k(entry(pos));
    int e_next = steps > 1 ? entry(pos + kBN) : 0;

    // the queries: B of the scores' product, columns permuted as K's are
    uint32_t qb[NT][kC][8];
    float qf[NT][2];  // score factors of rows 2t, 2t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint4 x[kC][2];
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[c][h] = make_uint4(0u, 0u, 0u, 0u);
          if (8 * n + g < p.group)
            x[c][h] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.query) + it.q.e.q0 * p.q_stride_t +
                                                      int64_t(it.kvh * p.group + 8 * n + g) * p.q_stride_h + 64 * c +
                                                      16 * t + 8 * h);
        }
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float f[8];
          Chunk<BF16>::expand(x[c][h], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int shift = i8::query_shift(top);
      const float s = i8::power(shift), f = p.qk_scale_log2 * i8::power(-shift);
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float y[8];
          Chunk<BF16>::expand(x[c][h], y);
#pragma unroll
          for (int i = 0; i < 4; ++i) qb[n][c][4 * h + i] = half2_bits(y[2 * i] * s, y[2 * i + 1] * s);
        }
      qf[n][0] = __shfl_sync(0xffffffffu, f, 8 * t);
      qf[n][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }

    float m[NT][2], l[NT][2];  // of rows 2t, 2t + 1 (l: this lane's tokens)
    float o[NT][2 * kW][4];    // O^T: see the products
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * kW; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }

#pragma unroll 1
    for (int j = 0; j < steps; ++j, pos += kBN) {
      const int pos0 = pos - lane;
      if (pos0 >= L) break;  // (the last tile: nothing for this warp)
      // V rows 2t, 2t + 1, 2t + 8, 2t + 9 of 16 tokens, D / 8 codes from D / 8 g on
      uint32_t v[2][4][kW];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (two tokens share a block)
          const unsigned char* src = vc + __shfl_sync(0xffffffffu, row, 16 * u + 8 * h + 2 * t) + 4 * kW * g;
          load_words(src, v[u][2 * h]);
          load_words(src + D, v[u][2 * h + 1]);
        }
      // S^T: tokens 16 u + g, + 8; rows 2t, 2t + 1
      float s[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const uint32_t x[4] = {kreg[u][0][c].x, kreg[u][0][c].y, kreg[u][0][c].z, kreg[u][0][c].w};
          const uint32_t y[4] = {kreg[u][1][c].x, kreg[u][1][c].y, kreg[u][1][c].z, kreg[u][1][c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 a = i8::widen4(x[i]), b = i8::widen4(y[i]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma(s[u][n], a.x, b.x, a.y, b.y, qb[n][c][2 * i], qb[n][c][2 * i + 1]);
          }
        }
      }
      // the scales of the lane's tokens 16 u + 8 h + g, and the value scales' exponents
      float tk[2][2], tv[2][2], ex[2][2];
      const float vex = i8::scale_exponent(vs);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tk[u][h] = __shfl_sync(0xffffffffu, ks, 16 * u + 8 * h + g);
          tv[u][h] = __shfl_sync(0xffffffffu, vs, 16 * u + 8 * h + g);
          ex[u][h] = __shfl_sync(0xffffffffu, vex, 16 * u + 8 * h + g);
        }
      const bool cut = pos0 + 32 > L || pos0 < lo;  // some token is not attended to
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
          if (hidden) tv[u][h] = 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& z = s[u][n][2 * h + r];
              z = hidden ? -INFINITY : z * (tk[u][h] * qf[n][r]);  // (no factor alone takes it out of range)
              move |= z + ex[u][h] > m[n][r] + kGap;
            }
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float a[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float mx = fmaxf(fmaxf(s[0][n][r] + ex[0][0], s[0][n][2 + r] + ex[0][1]),
                             fmaxf(s[1][n][r] + ex[1][0], s[1][n][2 + r] + ex[1][1]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const bool go = mx > m[n][r] + kGap || (m[n][r] == -INFINITY && mx > -INFINITY);
            a[r] = go ? fast_exp2(m[n][r] - mx) : 1.f;  // (0 from -infinity)
            if (go) m[n][r] = mx;
            l[n][r] *= a[r];
          }
#pragma unroll
          for (int i = 0; i < 2 * kW; ++i) {
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
        const float r0 = m[n][0] == -INFINITY ? 0.f : m[n][0] - i8::kTopWeight;
        const float r1 = m[n][1] == -INFINITY ? 0.f : m[n][1] - i8::kTopWeight;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float x = fast_exp2(s[u][n][2 * h] - r0), y = fast_exp2(s[u][n][2 * h + 1] - r1);
            l[n][0] += x;
            l[n][1] += y;
            pb[u][n][h] = transpose8x8(half2_bits(x * tv[u][h], y * tv[u][h]));
          }
      }
      // O^T: two products for each of the lane's words of V, whose first 8 rows are the lanes'
      // columns 4 w (then 4 w + 2), and the others the columns after them
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          uint32_t lo01[2], hi01[2];  // codes of columns 0, 1 and 2, 3 of two tokens, side by side
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = i8::flip4(v[u][2 * h][w]), y = i8::flip4(v[u][2 * h + 1][w]);
            lo01[h] = __byte_perm(x, y, 0x5140);
            hi01[h] = __byte_perm(x, y, 0x7362);
          }
          const uint2 a = i8::widen4_flipped(lo01[0]), b = i8::widen4_flipped(lo01[1]);
          const uint2 c = i8::widen4_flipped(hi01[0]), d = i8::widen4_flipped(hi01[1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma(o[n][2 * w], a.x, a.y, b.x, b.y, pb[u][n][0], pb[u][n][1]);
            mma(o[n][2 * w + 1], c.x, c.y, d.x, d.y, pb[u][n][0], pb[u][n][1]);
          }
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
        for (int w = 0; w < kW; ++w)
          *reinterpret_cast<float4*>(&sh.o[warp][8 * n + 2 * t + r][4 * kW * g + 4 * w]) =
              make_float4(o[n][2 * w][r], o[n][2 * w][2 + r], o[n][2 * w + 1][r], o[n][2 * w + 1][2 + r]);
      }
    }
    __syncthreads();
    constexpr int kPer = kThreads / kRows;  // threads of a row
    const int r = tid / kPer, c0 = tid % kPer;
    if (r < p.group) {
      float M = -INFINITY, den = 0.f, f[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.m[w][r]);
      const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        // (a warp whose scores are all NaN has no maximum: it counts as it stands)
        f[w] = sh.m[w][r] == -INFINITY ? 1.f : fast_exp2(sh.m[w][r] - ref);
        den += sh.l[w][r] * f[w];
      }
      const bool whole = it.begins() && it.ends();
      const float inv = !whole ? 1.f : den != 0.f ? 1.f / den : 0.f;
      const int64_t prow = int64_t(2 * blockIdx.x + (it.begins() ? 1 : 0)) * sp.rows + r;
      if (!whole && c0 == 0) sp.ml[prow] = make_float2(M, den);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + it.q.e.q0 * p.out_stride_t +
                           int64_t(it.kvh * p.group + r) * p.out_stride_h;
#pragma unroll
      for (int c = 4 * c0; c < D; c += 4 * kPer) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(&sh.o[w][r][c]);
          y = make_float4(y.x + x.x * f[w], y.y + x.y * f[w], y.z + x.z * f[w], y.w + x.w * f[w]);
        }
        y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
        if (!whole) {
          *reinterpret_cast<float4*>(sp.o + prow * D + c) = y;
        } else {
          const __nv_bfloat162 a = __floats2bfloat162_rn(y.x, y.y), b = __floats2bfloat162_rn(y.z, y.w);
          if (sp.out_vec) {
            *reinterpret_cast<uint2*>(out + c) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
          } else {
            out[c] = a.x;
            out[c + 1] = a.y;
            out[c + 2] = b.x;
            out[c + 3] = b.y;
          }
        }
      }
    }
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

}  // namespace decode_i8

namespace {

template <int D, int NT>
cudaError_t launch_decode_i8_tpl(const TreeParams& p, const TreeSplit& sp, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sp.grid));
  cfg.blockDim = dim3(decode_i8::kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, decode_i8::decode_i8_kernel<D, NT>, p, sp);
  note_launch();
  if (e != cudaSuccess) return e;
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_tree_merge(p, sp, stream);
}

}  // namespace

// Up to two tiles of 8 heads: a third would not leave registers for a step's codes.  64 sequences
// of 129 to 2048 positions with this kernel and with tree_i8.cu's: 8 KV heads of 4 heads of 128 36
// and 102 us, 4 KV heads of 16 29 and 53, 8 KV heads of 16 heads of 64 33 and 90.
bool decode_i8_supported(const TreeParams& p) {
  return !p.query_start_loc && p.group <= 16 && tree_i8_supported(p);
}

// What the registers allow (168 a thread; 255 with two tiles).  Batch and long contexts with two
// blocks of one tile 44 and 115 us, with three 38 and 97 (64 bytes a thread are spilled for heads
// of 128), with four (128 registers, many more spilled) 49 and 132.
int decode_i8_blocks_per_sm(int group) { return group <= 8 ? 3 : 2; }

cudaError_t launch_decode_i8(const TreeParams& p, TreeSplit sp, cudaStream_t stream) {
  sp.item_nodes = sp.tq = 1;
  if (p.head_dim == 128)
    return p.group <= 8 ? launch_decode_i8_tpl<128, 1>(p, sp, stream) : launch_decode_i8_tpl<128, 2>(p, sp, stream);
  return p.group <= 8 ? launch_decode_i8_tpl<64, 1>(p, sp, stream) : launch_decode_i8_tpl<64, 2>(p, sp, stream);
}

}  // namespace pkv
