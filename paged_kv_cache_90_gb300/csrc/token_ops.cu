// token_ops.cu — per-token passes between the activations and the paged cache: rotary
// positions with the cache write (rotary_and_cache), the write into a token-scaled
// 8-bit cache (quantize_and_cache), and the read back (read_cache).
//
// All are streams: every byte is touched once, so HBM bounds the large calls and the
// launch the small ones.  A head row (head_dim elements) is held by head_dim / 8
// neighbouring lanes, eight columns each, so that a row's largest magnitude is a few
// shuffles away and loads are 16 bytes wide.  The write with rotation and the one
// without are the same kernel.
#include "device_common.cuh"
#include "token_internal.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load_row8(const void* base, int64_t elt, float* f);
template <>
__device__ __forceinline__ void load_row8<BF16>(const void* base, int64_t elt, float* f) {
  Chunk<BF16>::expand(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elt), f);
}
template <>
__device__ __forceinline__ void load_row8<F32>(const void* base, int64_t elt, float* f) {
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + elt);
  const uint4 a = s[0], b = s[1];
  Chunk<F32>::expand(a, f);
  Chunk<F32>::expand(b, f + 4);
}

template <typename T>
__device__ __forceinline__ float load_one(const void* base, int64_t elt);
template <>
__device__ __forceinline__ float load_one<BF16>(const void* base, int64_t elt) {
  return bf16_lo_to_f32(static_cast<const uint16_t*>(base)[elt]);
}
template <>
__device__ __forceinline__ float load_one<F32>(const void* base, int64_t elt) {
  return static_cast<const float*>(base)[elt];
}

template <typename T>
__device__ __forceinline__ void store_row8(void* base, int64_t elt, const float* f);
template <>
__device__ __forceinline__ void store_row8<BF16>(void* base, int64_t elt, const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elt) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store_row8<F32>(void* base, int64_t elt, const float* f) {
  float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + elt);
  d[0] = make_float4(f[0], f[1], f[2], f[3]);
  d[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Eight values -> eight codes clamp(rint(x / s), +-127), s = amax / 127 (see pkv.h).
__device__ __forceinline__ uint2 quantize8(const float* x, float s) {
  uint32_t w[2] = {0u, 0u};
  if (s > 0.f) {  // (0: all zeros; NaN: zeros, the scale tells)
    const DivRn div(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int c = __float2int_rn(div(x[i]));
      c = min(127, max(-127, c));
      w[i >> 2] |= uint32_t(c & 0xff) << (8 * (i & 3));
    }
  }
  return make_uint2(w[0], w[1]);
}

// The scale of a row with largest magnitude `top`; `bad`: it holds an infinity or a NaN.
__device__ __forceinline__ float token_scale(float top, bool bad) {
  const float s = __fdiv_rn(top, 127.f);
  return bad ? __uint_as_float(0x7fc00000u) : s >= 0x1p-126f ? s : 0.f;
}

// One thread block per token (and, when few tokens leave SMs idle, per slice of its
// rows): query rows, then key rows, then value rows.
//
// The angle of pair i is position * turns[i] mod 2^64 in units of 2^-64 turn: a 64-bit
// product that wraps at whole turns, exact but for the 2^-53 relative error of the
// frequency, at any position.  Its top 32 bits, a signed fraction of a turn, go to
// sincospif: the cosines are within 3e-7 whatever the position, where a binary32 angle
// in radians would lose all its bits past 2^24.
template <typename Src, int D>
__global__ void __launch_bounds__(kThreads) token_write_kernel(const __grid_constant__ TokenParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // as in the other cache writes
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kLanes = D / 8;                // lanes per row
  constexpr int kRows = kThreads / kLanes;     // rows per pass
  __shared__ float2 cs[D / 2];                 // (cos, sin) of the token's pairs, times the magnitude
  const int64_t t = blockIdx.x;
  const int half = p.rotary_dim / 2;
  if (half) {
    if (threadIdx.x < half) {
      const int64_t pos = p.positions64 ? static_cast<const int64_t*>(p.positions)[t]
                                        : static_cast<const int32_t*>(p.positions)[t];
      const uint64_t turn = uint64_t(pos) * p.turns[threadIdx.x];
      const int32_t frac = int32_t(uint32_t(turn >> 32));  // 2^-32 turn, in [-1/2, 1/2)
      float s, c;
      sincospif(float(frac) * 0x1p-31f, &s, &c);
      cs[threadIdx.x] = make_float2(c * p.magnitude, s * p.magnitude);
    }
    __syncthreads();
  }
  const int64_t slot = p.w.slot_mapping[t];
  const bool in_cache = slot >= 0 && slot < p.w.num_blocks * p.w.block_size;
  if (slot >= 0 && !in_cache && threadIdx.x == 0 && blockIdx.y == 0) raise_device_error(p.w.err, kErrSlot);
  const int64_t blk = in_cache ? slot / p.w.block_size : 0;
  const int off = in_cache ? int(slot - blk * p.w.block_size) : 0;
  const int hq = p.num_heads, hk = p.w.num_kv_heads;
  const int rows = hq + (in_cache ? 2 * hk : 0);
  const int col = int(threadIdx.x % kLanes) * 8;
  // (a warp's lanes hold whole rows and take the same number of passes, for the shuffles)
  for (int base = int(blockIdx.y) * kRows; base < rows; base += int(gridDim.y) * kRows) {
    const int r = base + int(threadIdx.x) / kLanes;
    const bool live = r < rows;
    const bool is_q = r < hq, is_v = r >= hq + hk;
    const int h = is_q ? r : is_v ? r - hq - hk : r - hq;
    const void* src = is_q ? p.query : is_v ? p.w.value : p.w.key;
    const int64_t row = is_q ? t * p.q_stride_t + h * p.q_stride_h : t * p.w.src_stride_t + h * p.w.src_stride_h;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) load_row8<Src>(src, row + col, x);
    if (live && !is_v && col < p.rotary_dim) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          if (col + i < p.rotary_dim) {
            const float2 a = cs[(col + i) >> 1];
            const float lo = x[i], hi = x[i + 1];
            x[i] = lo * a.x - hi * a.y;
            x[i + 1] = hi * a.x + lo * a.y;
          }
        }
      } else {
        // the other column of each pair: half a rotary_dim away, 16-byte aligned when
        // half of it is a multiple of 8
        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if ((half & 7) == 0) {
          load_row8<Src>(src, row + (col < half ? col + half : col - half), y);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = col + i;
            if (c < p.rotary_dim) y[i] = load_one<Src>(src, row + (c < half ? c + half : c - half));
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = col + i;
          if (c < p.rotary_dim) {
            const float2 a = cs[c < half ? c : c - half];
            x[i] = x[i] * a.x + (c < half ? -y[i] : y[i]) * a.y;
          }
        }
      }
    }
    __syncwarp();  // every lane has read its row before one is written (query_out may be query)
    if (is_q) {
      if (live) store_row8<Src>(p.query_out, t * p.qo_stride_t + h * p.qo_stride_h + col, x);
    }
    if (p.w.cache_dtype == kI8) {
      float top = 0.f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        top = fmaxf(top, fabsf(x[i]));
        bad |= !(fabsf(x[i]) <= 3.402823466e38f);
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        bad |= __shfl_xor_sync(0xffffffffu, int(bad), o) != 0;
      }
      if (live && !is_q) {
        const float s = token_scale(top, bad);
        unsigned char* dst = static_cast<unsigned char*>(is_v ? p.w.value_cache : p.w.key_cache);
        *reinterpret_cast<uint2*>(dst + blk * p.w.cs_block + h * p.w.cs_head + off * D + col) = quantize8(x, s);
        if (col == 0) (is_v ? p.v_token_scales : p.k_token_scales)[blk * p.ts_block + h * p.ts_head + off] = s;
      }
    } else if (live && !is_q) {
      void* dst = is_v ? p.w.value_cache : p.w.key_cache;
      const int64_t at = blk * p.w.cs_block + h * p.w.cs_head + int64_t(off) * D + col;
      if (p.w.cache_dtype == kE4M3) {
        const float* hs = is_v ? p.w.v_head_scales : p.w.k_head_scales;
        const float s = hs ? __ldg(hs + h) : is_v ? p.w.v_scale : p.w.k_scale;
        *reinterpret_cast<uint2*>(static_cast<unsigned char*>(dst) + at) = e4m3_quantize8(x, DivRn(s));
      } else {
        store_row8<Src>(dst, at, x);
      }
    }
  }
}

// One thread per eight columns of a (token, tensor, KV head) row.
template <typename Dst, int D>
__global__ void __launch_bounds__(kThreads) token_read_kernel(const __grid_constant__ TokenParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kLanes = D / 8;
  const int64_t t = blockIdx.x;
  const int64_t slot = p.w.slot_mapping[t];
  if (slot < 0) return;
  if (slot >= p.w.num_blocks * p.w.block_size) {
    if (threadIdx.x == 0 && blockIdx.y == 0) raise_device_error(p.w.err, kErrSlot);
    return;
  }
  const int64_t blk = slot / p.w.block_size;
  const int off = int(slot - blk * p.w.block_size);
  const int hk = p.w.num_kv_heads;
  const int col = int(threadIdx.x % kLanes) * 8;
  constexpr int kRows = kThreads / kLanes;
  for (int r = int(blockIdx.y) * kRows + int(threadIdx.x) / kLanes; r < 2 * hk; r += int(gridDim.y) * kRows) {
    const bool is_v = r >= hk;
    const int h = is_v ? r - hk : r;
    const void* src = is_v ? p.w.value_cache : p.w.key_cache;
    const int64_t at = blk * p.w.cs_block + h * p.w.cs_head + int64_t(off) * D + col;
    float x[8];
    if (p.w.cache_dtype == kF32) {
      load_row8<F32>(src, at, x);
    } else if (p.w.cache_dtype == kBF16) {
      load_row8<BF16>(src, at, x);
    } else {
      const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(src) + at);
      float s;
      if (p.w.cache_dtype == kE4M3) {
        e4m3x4_to_f32x4(c.x, x);
        e4m3x4_to_f32x4(c.y, x + 4);
        const float* hs = is_v ? p.w.v_head_scales : p.w.k_head_scales;
        s = hs ? __ldg(hs + h) : is_v ? p.w.v_scale : p.w.k_scale;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = float(int(int8_t((i < 4 ? c.x : c.y) >> (8 * (i & 3)))));
        s = (is_v ? p.v_token_scales : p.k_token_scales)[blk * p.ts_block + h * p.ts_head + off];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= s;
    }
    void* dst = const_cast<void*>(is_v ? p.w.value : p.w.key);
    store_row8<Dst>(dst, t * p.w.src_stride_t + h * p.w.src_stride_h + col, x);
  }
}

// grid.y slices of a token's rows: one block per token once that fills the GPU
unsigned row_slices(int64_t tokens, int rows, int head_dim) {
  const int per_pass = kThreads / (head_dim / 8);
  const int passes = (rows + per_pass - 1) / per_pass;
  int64_t y = 1;
  while (y < passes && tokens * y < 608) ++y;  // 608 = 152 SMs x 4 blocks
  return unsigned(y);
}

template <typename K>
cudaError_t launch(K kern, const TokenParams& p, int rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.w.num_tokens), row_slices(p.w.num_tokens, rows, p.w.head_dim));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_write(const TokenParams& p, cudaStream_t stream) {
  const int rows = p.num_heads + 2 * p.w.num_kv_heads;
  if (p.w.src_dtype == kBF16)
    return p.w.head_dim == 128 ? launch(token_write_kernel<BF16, 128>, p, rows, stream)
                               : launch(token_write_kernel<BF16, 64>, p, rows, stream);
  return p.w.head_dim == 128 ? launch(token_write_kernel<F32, 128>, p, rows, stream)
                             : launch(token_write_kernel<F32, 64>, p, rows, stream);
}

cudaError_t launch_token_read(const TokenParams& p, cudaStream_t stream) {
  const int rows = 2 * p.w.num_kv_heads;
  if (p.w.src_dtype == kBF16)
    return p.w.head_dim == 128 ? launch(token_read_kernel<BF16, 128>, p, rows, stream)
                               : launch(token_read_kernel<BF16, 64>, p, rows, stream);
  return p.w.head_dim == 128 ? launch(token_read_kernel<F32, 128>, p, rows, stream)
                             : launch(token_read_kernel<F32, 64>, p, rows, stream);
}

}  // namespace pkv
