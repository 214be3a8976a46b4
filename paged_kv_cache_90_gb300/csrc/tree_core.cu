// tree_core.cu — attention of drafted trees and decode over a token-scaled cache on the
// CUDA cores: the path for what the tensor-core kernels do not take (f32 queries, f32 and
// e4m3 caches, bf16 caches of block sizes 2 and 4, groups of more than 128 query heads, a
// scale that is not above zero, rows not aligned to 16 bytes).
//
// One thread block per (query row, query head).  Its four warps take 32 keys at a time in
// turn: a lane computes one key's score from 16-byte loads of the key's row, then every
// lane owns head_dim / 32 output columns and the warp walks the 32 values.  Each warp
// keeps a running base-2 maximum, sum and output in binary32; the four are folded at the
// end.  Keys that the row does not attend to are not read.  Bound by the load latency of
// one key row per lane and by re-reading the keys for every head of a group; it is a
// path for rare types, not a fast one: 64 trees of 5 to 24 nodes over 160 to 2048 positions
// take 3.4 ms here (bf16), 62 us on the tensor cores.
#include "tree_common.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;

struct I8 { static constexpr int bytes = 1; };

template <typename KV>
__device__ __forceinline__ void expand16(const uint4& v, float* f) { Chunk<KV>::expand(v, f); }
template <>
__device__ __forceinline__ void expand16<I8>(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = float(int(int8_t(w[i >> 2] >> (8 * (i & 3)))));
}

template <typename KV>
__device__ __forceinline__ float value_at(const void* base, int64_t elt);
template <>
__device__ __forceinline__ float value_at<F32>(const void* b, int64_t e) { return static_cast<const float*>(b)[e]; }
template <>
__device__ __forceinline__ float value_at<BF16>(const void* b, int64_t e) {
  return bf16_lo_to_f32(static_cast<const uint16_t*>(b)[e]);
}
template <>
__device__ __forceinline__ float value_at<E4M3>(const void* b, int64_t e) {
  float f[4];
  e4m3x4_to_f32x4(static_cast<const uint8_t*>(b)[e], f);
  return f[0];
}
template <>
__device__ __forceinline__ float value_at<I8>(const void* b, int64_t e) {
  return float(int(static_cast<const int8_t*>(b)[e]));
}

template <typename KV, int D>
__global__ void __launch_bounds__(kWarps * 32) tree_core_kernel(const __grid_constant__ TreeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kCols = D / 32;
  __shared__ float q_sh[D];
  __shared__ float o_sh[kWarps][D];
  __shared__ float2 ml_sh[kWarps];
  const int t = int(blockIdx.x), h = int(blockIdx.y);
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  bool bad;
  if (h == 0 && threadIdx.x == 0)  // every sequence is checked, those whose rows are none of the batch's too
    for (int c = t; c < p.num_seqs; c += int(gridDim.x)) {
      (void)tree::extent(p, c, &bad);
      if (bad) raise_device_error(p.err, kErrContextLen);
    }
  // the row's sequence: the last one that starts at or before it
  int s = t;
  if (p.query_start_loc) {
    int a = 0, b = p.num_seqs;  // qsl[a] <= t < qsl[b], taking qsl[num_seqs] as the end
    if (t >= __ldg(p.query_start_loc + b)) return;  // behind the last sequence
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (__ldg(p.query_start_loc + m) <= t) a = m; else b = m;
    }
    s = a;
  }
  const tree::Extent e = tree::extent(p, s, &bad);
  const int node = t - e.q0;
  if (node < 0 || node >= e.n) return;
  const int64_t* mask = p.tree_mask ? p.tree_mask + int64_t(t) * p.mask_stride : nullptr;
  const int kvh = h / p.group;
  const float ks = p.k_head_scales ? __ldg(p.k_head_scales + kvh) : 1.f;
  if (threadIdx.x < D) {
    const int64_t at = int64_t(t) * p.q_stride_t + int64_t(h) * p.q_stride_h + threadIdx.x;
    const float q = p.q_dtype == kF32 ? static_cast<const float*>(p.query)[at]
                                      : bf16_lo_to_f32(static_cast<const uint16_t*>(p.query)[at]);
    q_sh[threadIdx.x] = q * (p.qk_scale_log2 * ks);
  }
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) o[c] = 0.f;
  for (int j0 = e.lo + 32 * warp; j0 < e.L; j0 += 32 * kWarps) {
    const int j = j0 + lane;
    bool on = j < e.L && (j < e.P || tree::sees_node(mask, j - e.P));
    int64_t at = 0;
    float z = -INFINITY, vs = 1.f;
    if (on) {
      const int lb = j / p.block_size, off = j - lb * p.block_size;
      int blk = __ldg(p.block_tables + int64_t(s) * p.bt_stride + lb);
      if (blk < 0 || int64_t(blk) >= p.num_blocks) {
        raise_device_error(p.err, kErrTableEntry);
        blk = 0;
      }
      at = int64_t(blk) * p.cs_block + int64_t(kvh) * p.cs_head + int64_t(off) * D;
      const uint4* row = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.key_cache) + at * KV::bytes);
      constexpr int kPer = 16 / KV::bytes;
      float acc = 0.f;
#pragma unroll 4
      for (int c = 0; c < D / kPer; ++c) {
        float f[kPer];
        expand16<KV>(row[c], f);
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc = fmaf(f[i], q_sh[c * kPer + i], acc);
      }
      if (p.k_token_scales) {
        const int64_t sc = int64_t(blk) * p.ts_block + int64_t(kvh) * p.ts_head + off;
        acc *= __ldg(p.k_token_scales + sc);
        vs = __ldg(p.v_token_scales + sc);
      }
      z = acc;
    }
    // (a NaN score must reach the output: the maximum skips it, the weight below does not)
    float top = z;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float m2 = fmaxf(m, top);
    const float ref = m2 == -INFINITY ? 0.f : m2;
    const float alpha = fast_exp2(m - ref);  // (0 while m is -infinity)
    const float w = on ? fast_exp2(z - ref) : 0.f;
    float sum = w;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * alpha + sum;
    m = m2;
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[c] *= alpha;
    unsigned todo = __ballot_sync(0xffffffffu, on);
    while (todo) {
      const int k = __ffs(int(todo)) - 1;
      todo &= todo - 1;
      const float wk = __shfl_sync(0xffffffffu, w * vs, k);
      const int64_t ak = __shfl_sync(0xffffffffu, at, k) + lane;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[c] = fmaf(wk, value_at<KV>(p.value_cache, ak + 32 * c), o[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < kCols; ++c) o_sh[warp][lane + 32 * c] = o[c];
  if (lane == 0) ml_sh[warp] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x >= D) return;
  float M = -INFINITY;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml_sh[w].x);
  const float ref = M == -INFINITY ? 0.f : M;
  float den = 0.f, num = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    const float x = fast_exp2(ml_sh[w].x - ref);
    den = fmaf(ml_sh[w].y, x, den);
    num = fmaf(o_sh[w][threadIdx.x], x, num);
  }
  const float vh = p.v_head_scales ? __ldg(p.v_head_scales + kvh) : p.v_scale;
  const float res = den != 0.f ? num / den * vh : 0.f;  // (no key attended to: zero)
  const int64_t at = int64_t(t) * p.out_stride_t + int64_t(h) * p.out_stride_h + threadIdx.x;
  if (p.q_dtype == kF32)
    static_cast<float*>(p.out)[at] = res;
  else
    static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(res);
}

template <typename KV>
cudaError_t launch_kv(const TreeParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.num_tokens), unsigned(p.num_heads));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = p.head_dim == 128 ? cudaLaunchKernelEx(&cfg, tree_core_kernel<KV, 128>, p)
                                          : cudaLaunchKernelEx(&cfg, tree_core_kernel<KV, 64>, p);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_core(const TreeParams& p, cudaStream_t stream) {
  switch (p.kv_dtype) {
    case kF32: return launch_kv<F32>(p, stream);
    case kBF16: return launch_kv<BF16>(p, stream);
    case kE4M3: return launch_kv<E4M3>(p, stream);
    default: return launch_kv<I8>(p, stream);
  }
}

}  // namespace pkv
