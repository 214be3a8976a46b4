// decode_few.cuh — what the decode kernels of few query heads a KV head (decode_i8.cu,
// decode_e2m1.cu) share: loads and products from registers, and the fold of a block's warps.
//
// Both take the small transposed products (mma m16n8k16, tokens or columns x heads), whose A operand
// is widened in registers; a warp keeps its own reference, sums and O^T of its positions, and the
// four warps are folded at an item's end, in order.
#pragma once

#include "i8_codes.cuh"
#include "tree_split.cuh"

namespace pkv {
namespace decode_few {

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
  tree::Range range;
  longlong2 warp_sum[kWarps];
  float m[kWarps][8 * NT], l[kWarps][8 * NT];
};
// The warps' O, row by row, at an item's end.
template <int D, int NT>
struct alignas(16) Rows {
  float o[kWarps][8 * NT][D + 4];
};

// The warps' results in `sh` and `rows` together: row r of the item to the output, or to its part.  `factor`:
// the cache's on the values.
template <int D, int NT>
__device__ __forceinline__ void fold_warps(const TreeParams& p, const TreeSplit& sp, const tree::Walk& it,
                                           const Shared<D, NT>& sh, const Rows<D, NT>& rows, float factor) {
  const int tid = threadIdx.x;
  constexpr int kPer = kThreads / (8 * NT);  // threads of a row
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
    const float inv = (!whole ? 1.f : den != 0.f ? 1.f / den : 0.f) * factor;
    const int64_t prow = int64_t(2 * blockIdx.x + (it.begins() ? 1 : 0)) * sp.rows + r;
    if (!whole && c0 == 0) sp.ml[prow] = make_float2(M, den);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + it.q.e.q0 * p.out_stride_t +
                         int64_t(it.kvh * p.group + r) * p.out_stride_h;
#pragma unroll
    for (int c = 4 * c0; c < D; c += 4 * kPer) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&rows.o[w][r][c]);
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
}

}  // namespace decode_few
}  // namespace pkv
