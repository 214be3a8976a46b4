// token_ops.cu — per-token passes between the activations and the paged cache: rotary
// positions with the cache write (rotary_and_cache), the write into a token-scaled
// 8-bit cache or a 4-bit one (quantize_and_cache), and the read back (read_cache).
//
// All are streams: every byte is touched once, so HBM bounds the large calls and the
// launch the small ones.  A head row (head_dim elements) is held by head_dim / 8
// neighbouring lanes, eight columns each, so that a row's largest magnitude is a few
// shuffles away and loads are 8 or 16 bytes wide.  A warp takes a slice of one token's rows,
// four passes' loads at a time, and waits for nothing else before them (not for the slot).
//
// What it measured: rotary write of 16384 tokens of 32 + 2 x 8 heads of 128 in bf16 (403 MB)
// 71 us, 5.7 TB/s (a block per token with the cosines in shared memory: 175 us); quantising
// write of 16384 tokens of 2 x 8 heads 31 us, read back into f32 26 us (168 MB, 6.4 TB/s).  The
// write is held back by its instructions, 190 for 8 columns of two rows, issued in four of five
// cycles.  Into a 4-bit cache the same write takes 19 us (86 MB; instructions in three of four
// cycles), read back into f32 27 us (153 MB, 5.6 TB/s; both over buffers that L2 does not hold); the
// rotary write with three position axes in turn over the pairs 73 us, 5.5 TB/s, and into a 4-bit
// cache, with one axis or three, 82 us (354 MB, 4.3 TB/s).
#include "device_common.cuh"
#include "e2m1_codes.cuh"
#include "token_internal.h"

namespace pkv {

namespace {

constexpr int kWarps = 4;     // of a block: a warp takes a slice of one token's rows
constexpr int kBatch = 4;     // passes whose loads a warp issues together (rotary write of a prefill
                              // step with 2, 4 and 8: 81, 75, 78 us; quantising 57, 57, 66 us)
constexpr int kFewRows = 48;  // rows of a slice at most (16, 24, 48: 83, 77, 73 us; see slices())

// A value that is the same in all lanes, so that the compiler knows it (and computes what
// follows from it once for the warp).
template <typename T>
__device__ __forceinline__ T one_answer(T x) { return __shfl_sync(0xffffffffu, x, 0); }

// How a row's columns go to its lanes, two groups of four each: side by side as pairs of
// columns turn (none, or 2 i with 2 i + 1), or one of each half of the rotated columns (i with
// half + i, half a multiple of 4); kOdd is the latter for any other half.
enum Layout { kPairs, kHalves, kOdd };

// What a rotary write does beside the common case, each kind compiled by itself: with the tests for
// both in one kernel a prefill step's write took 75 us instead of 71.  kFour is held back by its
// instructions: it makes a row's factor anew in every pass and a group's scale in two lanes, and brings
// all layouts' columns in order through shared memory (82 us where the bytes take 53).
enum Kind { kPlain, kAxes, kFour };  // several position axes; a 4-bit cache (with or without them)

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int kLanes>
__device__ __forceinline__ uint32_t row_top_bits(const float (&x)[8]) {
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top;
}

// A lane's eight columns as they are stored, so that a batch of loads takes few registers.
template <typename T>
struct Raw;
template <>
struct Raw<BF16> {
  uint2 a, b;
  // The bits of a row's largest magnitude, as a binary32 number's (all lanes of the row call).
  template <int kLanes>
  __device__ __forceinline__ uint32_t row_top() const {
    uint32_t m = max_u16x2(max_u16x2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu), max_u16x2(b.x & 0x7fff7fffu, b.y & 0x7fff7fffu));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return max(m & 0xffff0000u, m << 16);
  }
  __device__ __forceinline__ void load(const void* base, int64_t elt, int c0, int c1, bool joined) {
    const uint16_t* s = static_cast<const uint16_t*>(base) + elt;
    if (joined) {
      const uint4 v = *reinterpret_cast<const uint4*>(s + c0);
      a = make_uint2(v.x, v.y);
      b = make_uint2(v.z, v.w);
    } else {
      a = *reinterpret_cast<const uint2*>(s + c0);
      b = *reinterpret_cast<const uint2*>(s + c1);
    }
  }
  __device__ __forceinline__ void expand(float* f) const { Chunk<BF16>::expand(make_uint4(a.x, a.y, b.x, b.y), f); }
  __device__ __forceinline__ void clear() { a = b = make_uint2(0u, 0u); }
};
template <>
struct Raw<F32> {
  uint4 a, b;
  template <int kLanes>
  __device__ __forceinline__ uint32_t row_top() const {
    float f[8];
    expand(f);
    return row_top_bits<kLanes>(f);
  }
  __device__ __forceinline__ void load(const void* base, int64_t elt, int c0, int c1, bool) {
    const float* s = static_cast<const float*>(base) + elt;
    a = *reinterpret_cast<const uint4*>(s + c0);
    b = *reinterpret_cast<const uint4*>(s + c1);
  }
  __device__ __forceinline__ void expand(float* f) const {
    Chunk<F32>::expand(a, f);
    Chunk<F32>::expand(b, f + 4);
  }
  __device__ __forceinline__ void clear() { a = b = make_uint4(0u, 0u, 0u, 0u); }
};

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
__device__ __forceinline__ void store_row(void* base, int64_t elt, int c0, int c1, bool joined, const float* f);
template <>
__device__ __forceinline__ void store_row<BF16>(void* base, int64_t elt, int c0, int c1, bool joined, const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  uint16_t* d = static_cast<uint16_t*>(base) + elt;
  if (joined) {
    *reinterpret_cast<uint4*>(d + c0) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<uint2*>(d + c0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(d + c1) = make_uint2(w[2], w[3]);
  }
}
template <>
__device__ __forceinline__ void store_row<F32>(void* base, int64_t elt, int c0, int c1, bool, const float* f) {
  float* d = static_cast<float*>(base) + elt;
  *reinterpret_cast<float4*>(d + c0) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(d + c1) = make_float4(f[4], f[5], f[6], f[7]);
}

// Eight codes (words of columns c0 .. and c1 ..) to a row of an 8-bit cache.
__device__ __forceinline__ void store_codes(void* base, int64_t elt, int c0, int c1, bool joined, uint2 w) {
  unsigned char* d = static_cast<unsigned char*>(base) + elt;
  if (joined) {
    *reinterpret_cast<uint2*>(d + c0) = w;
  } else {
    *reinterpret_cast<uint32_t*>(d + c0) = w.x;
    *reinterpret_cast<uint32_t*>(d + c1) = w.y;
  }
}

// Eight values -> eight codes rint(x / s), s = amax / 127 correctly rounded, or 0 (all codes 0)
// or NaN (zeros too).  |x / s| is at most 127 (1 + 2^-23), so none needs clamping.
//
// The quotient is the correctly rounded one: the product with the correctly rounded 1 / s, and
// twice the remainder's share added (as DivRn; what underflows on the way belongs to quotients
// far below 1/2).  16-bit activations have many quotients in the middle of two codes: a cheaper
// quotient, with a division for those near it, divided in every second pass and was no faster.
__device__ __forceinline__ uint2 quantize8(const float* x, float s) {
  uint32_t c[8];
  if (s >= 0x1p-90f) {
    const float y = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float q = __fmul_rn(x[i], y);
      q = __fmaf_rn(__fmaf_rn(-s, q, x[i]), y, q);
      q = __fmaf_rn(__fmaf_rn(-s, q, x[i]), y, q);
      c[i] = __float_as_uint(__fadd_rn(q, 12582912.f));  // (1.5 * 2^23: rounded, in the low bits)
    }
  } else if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = uint32_t(__float2int_rn(__fdiv_rn(x[i], s)));
  } else {
    return make_uint2(0u, 0u);
  }
  const uint32_t a = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  const uint32_t b = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
  return make_uint2(a, b);
}

// The scale of a row whose largest magnitude has the bits `top` (an infinity's or a NaN's are
// above every number's).
__device__ __forceinline__ float token_scale(uint32_t top) {
  const DivRn div(127.f);
  const float s = div(__uint_as_float(top));
  return top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : s >= 0x1p-126f ? s : 0.f;
}

__device__ __forceinline__ uint64_t angle_at(int64_t pos, uint64_t turn, const uint32_t* low) {
  uint64_t angle = uint64_t(pos) * turn;
  if (pos != int32_t(pos)) angle += uint64_t((pos >> 32) * int64_t(*low)) + (uint64_t(uint32_t(pos)) * *low >> 32);
  return angle;
}

// The position that turns pair k of token t.
__device__ __forceinline__ int64_t axis_position(const TokenParams& p, int64_t t, int k) {
  const int64_t at = int64_t((p.axis[k >> 4] >> (2 * (k & 15))) & 3u) * p.pos_stride + t;
  return p.positions64 ? static_cast<const int64_t*>(p.positions)[at] : static_cast<const int32_t*>(p.positions)[at];
}

// A row's columns 8 l .. 8 l + 7 to a 4-bit cache: `codes` and `scales` are the row's first bytes,
// `top` the bits of its group's largest magnitude.  All lanes of the row call it (`live`: the row is
// stored); a group is two lanes', and its scales leave as words of four.
__device__ __forceinline__ void store_e2m1(const float (&x)[8], uint32_t top, const e2m1::Factor& f, unsigned char* codes,
                                           unsigned char* scales, int l, bool live) {
  const e2m1::Group g(top, f);
  uint32_t four = g.byte << (8 * ((l >> 1) & 3));
  four |= __shfl_xor_sync(0xffffffffu, four, 2);
  four |= __shfl_xor_sync(0xffffffffu, four, 4);
  if (!live) return;
  *reinterpret_cast<uint32_t*>(codes + 4 * l) = e2m1::encode8(x, g);
  if ((l & 7) == 0) *reinterpret_cast<uint32_t*>(scales + (l >> 1)) = four;
}

// The bits of a group's largest magnitude, as a binary32 number's: of 16 columns as they are stored.
template <typename Src, int N>
__device__ __forceinline__ uint32_t group_top(const uint4 (&raw)[N]) {
  constexpr uint32_t kMagnitude = Src::bytes == 2 ? 0x7fff7fffu : 0x7fffffffu;
  auto larger = [](uint32_t a, uint32_t b) { return Src::bytes == 2 ? max_u16x2(a, b) : max(a, b); };
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i)
    m = larger(m, larger(larger(raw[i].x & kMagnitude, raw[i].y & kMagnitude),
                         larger(raw[i].z & kMagnitude, raw[i].w & kMagnitude)));
  return Src::bytes == 2 ? max(m & 0xffff0000u, m << 16) : m;
}

__device__ __forceinline__ float cache_factor(const CacheWriteParams& w, bool is_v, int h) {
  const float* hs = is_v ? w.v_head_scales : w.k_head_scales;
  return hs ? __ldg(hs + h) : is_v ? w.v_scale : w.k_scale;
}

// One warp per slice of a token's rows: query rows, then key rows, then value rows.  Block
// (x, y): slice y of kWarps tokens.
//
// The angle of pair i is position * (turns[i] + turns_low[i] 2^-32) mod 2^64 in units of 2^-64
// turn: products of whole numbers that wrap at whole turns, off by 2^-34 turn at the farthest
// position (the low part is less than 2^-33 turn at those of 32 bits, and left out there: 70.9
// us in place of 71.3 for a prefill step's write, 70.0 without any).  Its top 32 bits, a signed
// fraction of a turn, go to sincospif as a binary32 number (24 of them, 1e-7 of a radian): the
// cosines are within 3e-7 whatever the position, where a binary32 angle in radians would lose
// all its bits past 2^24.  A lane has the same four pairs in every row, so their cosines and
// sines are in its registers.
template <typename Src, int D, Layout kLayout, Kind kKind>
__global__ void __launch_bounds__(32 * kWarps) token_write_kernel(const __grid_constant__ TokenParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows of a pass
  constexpr int kN = kLayout == kOdd ? 1 : kBatch;
  constexpr bool kJoined = kLayout != kHalves && (Src::bytes == 2 || kLayout == kOdd);  // 8 columns side by side
  __shared__ uint64_t turns[64];
  __shared__ alignas(16) float staged[kKind == kFour ? kWarps : 1][kKind == kFour ? 256 : 4];  // a pass's rows, columns in order
  const bool axes = kKind == kAxes || (kKind == kFour && p.num_axes);
  const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
  const int half = p.rotary_dim / 2;
  if (int(threadIdx.x) < half) turns[threadIdx.x] = p.turns[threadIdx.x];
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // as in the other cache writes
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t t = int64_t(blockIdx.x) * kWarps + one_answer(int(threadIdx.x) >> 5);
  if (t >= p.w.num_tokens) return;
  const int64_t slot = one_answer(p.w.slot_mapping[t]);
  int64_t pos = 0;
  if (half && !axes) pos = p.positions64 ? static_cast<const int64_t*>(p.positions)[t] : static_cast<const int32_t*>(p.positions)[t];
  int c0 = 8 * l, c1 = 8 * l + 4, pair0 = 0, pair1 = 0;  // (pairs of the first and last four columns)
  bool turning = false;
  if (kLayout == kHalves) {
    if (4 * l < half) {
      c0 = 4 * l;
      c1 = half + c0;
      pair0 = c0;
      pair1 = c0 + 2;
      turning = true;
    } else {
      c0 = p.rotary_dim + 8 * (l - half / 4);
      c1 = c0 + 4;
    }
  } else if (kLayout == kPairs) {
    if (!kJoined) {  // (so that a warp's 16-byte accesses lie side by side)
      c0 = 4 * l;
      c1 = D / 2 + 4 * l;
    }
    pair0 = c0 / 2;
    pair1 = c1 / 2;
  }
  float cs[4], sn[4];
  bool turn[4];
  const int hq = p.num_heads, hk = p.w.num_kv_heads;
  const int rows = hq + 2 * hk;
  const int passes = (rows + kRows - 1) / kRows, per = (passes + int(gridDim.y) - 1) / int(gridDim.y);
  const int first = int(blockIdx.y) * per, last = min(first + per, passes);
  // (all of a warp's lanes take the same passes, for the shuffles)
  for (int p0 = first; p0 < last; p0 += kN) {
    Raw<Src> raw[kN];
    float y[8];  // (kOdd) the other columns of the pairs
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      const int r = (p0 + u) * kRows + sub;
      raw[u].clear();
      if (p0 + u < last && r < rows) {
        const bool is_q = r < hq, is_v = r >= hq + hk;
        const void* src = is_q ? p.query : is_v ? p.w.value : p.w.key;
        const int64_t row = is_q ? t * p.q_stride_t + r * p.q_stride_h
                                 : t * p.w.src_stride_t + (is_v ? r - hq - hk : r - hq) * p.w.src_stride_h;
        raw[u].load(src, row, c0, c1, kJoined);
        if (kLayout == kOdd && !is_v) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = c0 + i;
            if (c < p.rotary_dim) y[i] = load_one<Src>(src, row + (c < half ? c + half : c - half));
          }
        }
      }
    }
    if (p0 == first && half && kLayout != kOdd) {  // (behind the first loads, as is all that needs the slot)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = (i < 2 ? pair0 : pair1 - 2) + i;
        turn[i] = kLayout == kHalves ? turning : k < half;
        const int64_t at = axes && turn[i] ? axis_position(p, t, k) : pos;
        const uint64_t angle = turn[i] ? angle_at(at, turns[k], p.turns_low + k) : 0;
        sincospif(float(int32_t(uint32_t(angle >> 32))) * 0x1p-31f, &sn[i], &cs[i]);  // 2^-32 turn, in [-1/2, 1/2)
        cs[i] *= p.magnitude;
        sn[i] *= p.magnitude;
      }
    }
    const bool in_cache = slot >= 0 && slot < p.w.num_blocks * p.w.block_size;
    const int64_t blk = in_cache ? slot >> (31 - __clz(p.w.block_size)) : 0;  // (a power of two)
    const int off = in_cache ? int(slot) & (p.w.block_size - 1) : 0;
    if (kLayout == kOdd) __syncwarp();  // every lane has read its row before one is written (query_out may be query)
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      if (p0 + u >= last) break;
      const int r = (p0 + u) * kRows + sub;
      const bool live = r < rows, is_q = r < hq, is_v = r >= hq + hk;
      const int h = is_q ? r : is_v ? r - hq - hk : r - hq;
      float x[8];
      raw[u].expand(x);
      if (half && !is_v) {
        if (kLayout == kOdd) {
          if (live) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              const int c = c0 + i;
              if (c >= p.rotary_dim) break;
              const int pair = c < half ? c : c - half;
              const int64_t at = axes ? axis_position(p, t, pair) : pos;
              const uint64_t angle = angle_at(at, turns[pair], p.turns_low + pair);
              float s, k;
              sincospif(float(int32_t(uint32_t(angle >> 32))) * 0x1p-31f, &s, &k);
              s *= p.magnitude;
              k *= p.magnitude;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (e == i) x[e] = x[e] * k + (c < half ? -y[e] : y[e]) * s;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& a = x[kLayout == kHalves ? i : 2 * i];
            float& b = x[kLayout == kHalves ? 4 + i : 2 * i + 1];
            const float lo = a, hi = b;
            if (turn[i]) {
              a = lo * cs[i] - hi * sn[i];
              b = hi * cs[i] + lo * sn[i];
            }
          }
        }
      }
      if (is_q) {
        if (live) store_row<Src>(p.query_out, t * p.qo_stride_t + h * p.qo_stride_h, c0, c1, kJoined, x);
      }
      void* dst = is_v ? p.w.value_cache : p.w.key_cache;
      if constexpr (kKind == kFour) {
        if ((p0 + u + 1) * kRows <= hq) continue;  // (query rows alone)
        float* row = staged[threadIdx.x >> 5] + sub * D;
        *reinterpret_cast<float4*>(row + c0) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(row + c1) = make_float4(x[4], x[5], x[6], x[7]);
        __syncwarp();
        const float4 a = *reinterpret_cast<const float4*>(row + 8 * l), b = *reinterpret_cast<const float4*>(row + 8 * l + 4);
        __syncwarp();
        const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const bool stored = live && !is_q && in_cache;
        store_e2m1(y, row_top_bits<2>(y), e2m1::Factor(stored ? cache_factor(p.w, is_v, h) : 1.f),
                   static_cast<unsigned char*>(dst) + blk * p.w.cs_block + h * p.w.cs_head + off * (D / 2),
                   (is_v ? p.v_group_scales : p.k_group_scales) + blk * p.ts_block + h * p.ts_head + off * (D / 16), l,
                   stored);
      } else {
        const int64_t at = blk * p.w.cs_block + h * p.w.cs_head + int64_t(off) * D;
        if (p.w.cache_dtype == kI8) {
          const uint32_t top = row_top_bits<kLanes>(x);
          if (live && !is_q && in_cache) {
            const float s = token_scale(top);
            store_codes(dst, at, c0, c1, kJoined, quantize8(x, s));
            if (l == 0) (is_v ? p.v_token_scales : p.k_token_scales)[blk * p.ts_block + h * p.ts_head + off] = s;
          }
        } else if (live && !is_q && in_cache) {
          if (p.w.cache_dtype == kE4M3) {
            const float* hs = is_v ? p.w.v_head_scales : p.w.k_head_scales;
            const float s = hs ? __ldg(hs + h) : is_v ? p.w.v_scale : p.w.k_scale;
            store_codes(dst, at, c0, c1, kJoined, e4m3_quantize8(x, DivRn(s)));
          } else {
            store_row<Src>(dst, at, c0, c1, kJoined, x);
          }
        }
      }
    }
  }
  if (slot >= p.w.num_blocks * p.w.block_size && lane == 0 && blockIdx.y == 0) raise_device_error(p.w.err, kErrSlot);
}

// The same for the write into a token-scaled cache alone: key rows, then value rows.
template <typename Src, int D>
__global__ void __launch_bounds__(32 * kWarps) token_quantize_kernel(const __grid_constant__ TokenParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  constexpr bool kJoined = Src::bytes == 2;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t t = int64_t(blockIdx.x) * kWarps + one_answer(int(threadIdx.x) >> 5);
  if (t >= p.w.num_tokens) return;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
  const int64_t slot = one_answer(p.w.slot_mapping[t]);
  const int c0 = kJoined ? 8 * l : 4 * l, c1 = kJoined ? c0 + 4 : c0 + D / 2;
  const int hk = p.w.num_kv_heads;
  // (a pass is of one tensor: the choice is the warp's, not a lane's)
  const int tensor = (hk + kRows - 1) / kRows, passes = 2 * tensor;
  const int per = (passes + int(gridDim.y) - 1) / int(gridDim.y);
  const int first = int(blockIdx.y) * per, last = min(first + per, passes);
  const int64_t from = t * p.w.src_stride_t;
  for (int p0 = first; p0 < last; p0 += kBatch) {
    Raw<Src> raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const bool is_v = p0 + u >= tensor;
      const int h = (p0 + u - (is_v ? tensor : 0)) * kRows + sub;
      raw[u].clear();
      if (p0 + u < last && h < hk) raw[u].load(is_v ? p.w.value : p.w.key, from + h * p.w.src_stride_h, c0, c1, kJoined);
    }
    if (slot < 0) return;  // padding
    if (slot >= p.w.num_blocks * p.w.block_size) {
      if (lane == 0 && blockIdx.y == 0) raise_device_error(p.w.err, kErrSlot);
      return;
    }
    const int64_t blk = slot >> (31 - __clz(p.w.block_size));
    const int off = int(slot) & (p.w.block_size - 1);
    const int64_t to = blk * p.w.cs_block + int64_t(off) * D, scale_to = blk * p.ts_block + off;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (p0 + u >= last) break;
      const bool is_v = p0 + u >= tensor;
      const int h = (p0 + u - (is_v ? tensor : 0)) * kRows + sub;
      const uint32_t top = raw[u].template row_top<kLanes>();
      if (h >= hk) continue;
      float x[8];
      raw[u].expand(x);
      const float s = token_scale(top);
      store_codes(is_v ? p.w.value_cache : p.w.key_cache, to + h * p.w.cs_head, c0, c1, kJoined, quantize8(x, s));
      if (l == 0) (is_v ? p.v_token_scales : p.k_token_scales)[scale_to + h * p.ts_head] = s;
    }
  }
}

// And into a 4-bit cache alone.  A lane has a group's 16 columns: its scale, a division and a
// reciprocal, is computed once and no lane waits for another's maximum: 15.4 M warp instructions
// for 16384 tokens of 2 x 8 heads in bf16 and 20.7 us (cold), with eight columns a lane 23.0 M and 26.8 us.
// Eight blocks an SM, for which 7 registers are spilled (write and read back 44.5 us; 45.4 with seven
// blocks, 45.5 with six; 45.1 with the loads of two passes together).
template <typename Src, int D>
__global__ void __launch_bounds__(32 * kWarps, 8) token_four_kernel(const __grid_constant__ TokenParams p) {
  constexpr int kPasses = kBatch * 2 / Src::bytes, kLanes = D / 16, kRows = 32 / kLanes, kLoads = Src::bytes;  // 16-byte loads of a group
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t t = int64_t(blockIdx.x) * kWarps + one_answer(int(threadIdx.x) >> 5);
  if (t >= p.w.num_tokens) return;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
  const int64_t slot = one_answer(p.w.slot_mapping[t]);
  const int hk = p.w.num_kv_heads;
  const int tensor = (hk + kRows - 1) / kRows, passes = 2 * tensor;  // (a pass is of one tensor)
  const int per = (passes + int(gridDim.y) - 1) / int(gridDim.y);
  const int first = int(blockIdx.y) * per, last = min(first + per, passes);
  const int64_t from = t * p.w.src_stride_t + 16 * l;
  const e2m1::Factor k_factor(p.w.k_scale), v_factor(p.w.v_scale);
  for (int p0 = first; p0 < last; p0 += kPasses) {
    uint4 raw[kPasses][kLoads];
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const bool is_v = p0 + u >= tensor;
      const int h = (p0 + u - (is_v ? tensor : 0)) * kRows + sub;
      const bool live = p0 + u < last && h < hk;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(is_v ? p.w.value : p.w.key) +
                                                        (from + h * p.w.src_stride_h) * Src::bytes);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) raw[u][i] = live ? src[i] : make_uint4(0u, 0u, 0u, 0u);
    }
    if (slot < 0) return;  // padding
    if (slot >= p.w.num_blocks * p.w.block_size) {
      if (lane == 0 && blockIdx.y == 0) raise_device_error(p.w.err, kErrSlot);
      return;
    }
    const int64_t blk = slot >> (31 - __clz(p.w.block_size));
    const int off = int(slot) & (p.w.block_size - 1);
    const int64_t to = blk * p.w.cs_block + off * (D / 2) + 8 * l, scale_to = blk * p.ts_block + off * (D / 16) + l;
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      if (p0 + u >= last) break;
      const bool is_v = p0 + u >= tensor;
      const int h = (p0 + u - (is_v ? tensor : 0)) * kRows + sub;
      e2m1::Factor f = is_v ? v_factor : k_factor;
      if (is_v ? p.w.v_head_scales != nullptr : p.w.k_head_scales != nullptr)
        f = e2m1::Factor(h < hk ? cache_factor(p.w, is_v, h) : 1.f);
      float x[16];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) Chunk<Src>::expand(raw[u][i], x + 16 / kLoads * i);
      const e2m1::Group g(group_top<Src>(raw[u]), f);
      uint32_t four = g.byte << (8 * (l & 3));  // (scales leave as words of four)
      four |= __shfl_xor_sync(0xffffffffu, four, 1);
      four |= __shfl_xor_sync(0xffffffffu, four, 2);
      if (h >= hk) continue;
      *reinterpret_cast<uint2*>(static_cast<unsigned char*>(is_v ? p.w.value_cache : p.w.key_cache) + to + h * p.w.cs_head) =
          make_uint2(e2m1::encode8(x, g), e2m1::encode8(x + 8, g));
      if ((l & 3) == 0)
        *reinterpret_cast<uint32_t*>((is_v ? p.v_group_scales : p.k_group_scales) + scale_to + h * p.ts_head) = four;
    }
  }
}

// The read back: a warp per slice of a token's key rows, then value rows.
template <typename Dst, int D, int type>
__global__ void __launch_bounds__(32 * kWarps) token_read_kernel(const __grid_constant__ TokenParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  constexpr bool kJoined = Dst::bytes == 2;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t t = int64_t(blockIdx.x) * kWarps + one_answer(int(threadIdx.x) >> 5);
  if (t >= p.w.num_tokens) return;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
  const int64_t slot = one_answer(p.w.slot_mapping[t]);
  if (slot < 0) return;
  if (slot >= p.w.num_blocks * p.w.block_size) {
    if (lane == 0 && blockIdx.y == 0) raise_device_error(p.w.err, kErrSlot);
    return;
  }
  const int64_t blk = slot >> (31 - __clz(p.w.block_size));
  const int off = int(slot) & (p.w.block_size - 1);
  const int hk = p.w.num_kv_heads;
  const int c0 = kJoined ? 8 * l : 4 * l, c1 = kJoined ? c0 + 4 : c0 + D / 2;
  const int tensor = (hk + kRows - 1) / kRows, passes = 2 * tensor;  // (a pass is of one tensor)
  const int per = (passes + int(gridDim.y) - 1) / int(gridDim.y);
  const int first = int(blockIdx.y) * per, last = min(first + per, passes);
  for (int p0 = first; p0 < last; p0 += kBatch) {
    uint4 a[kBatch], b[kBatch];  // columns c0 .. and c1 .., as they are stored
    float s[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const bool is_v = p0 + u >= tensor;
      const int h = (p0 + u - (is_v ? tensor : 0)) * kRows + sub;
      if (p0 + u >= last || h >= hk) continue;
      const int elt = type == kF32 ? 4 : type == kBF16 ? 2 : 1;
      const unsigned char* src = static_cast<const unsigned char*>(is_v ? p.w.value_cache : p.w.key_cache) +
                                 (blk * p.w.cs_block + h * p.w.cs_head + int64_t(off) * (type == kE2M1 ? D / 2 : D)) * elt;
      if (type == kE2M1) {
        const unsigned char* g = (is_v ? p.v_group_scales : p.k_group_scales) + blk * p.ts_block + h * p.ts_head + off * (D / 16);
        a[u].x = *reinterpret_cast<const uint16_t*>(src + c0 / 2);
        b[u].x = *reinterpret_cast<const uint16_t*>(src + c1 / 2);
        a[u].y = g[c0 >> 4];
        b[u].y = g[c1 >> 4];
        s[u] = cache_factor(p.w, is_v, h);
      } else if (type == kF32) {
        a[u] = *reinterpret_cast<const uint4*>(src + 4 * c0);
        b[u] = *reinterpret_cast<const uint4*>(src + 4 * c1);
      } else if (type == kBF16) {
        const uint2 x = *reinterpret_cast<const uint2*>(src + 2 * c0), y = *reinterpret_cast<const uint2*>(src + 2 * c1);
        a[u].x = x.x; a[u].y = x.y;
        b[u].x = y.x; b[u].y = y.y;
      } else {
        a[u].x = *reinterpret_cast<const uint32_t*>(src + c0);
        b[u].x = *reinterpret_cast<const uint32_t*>(src + c1);
        const float* hs = is_v ? p.w.v_head_scales : p.w.k_head_scales;
        s[u] = type == kI8 ? (is_v ? p.v_token_scales : p.k_token_scales)[blk * p.ts_block + h * p.ts_head + off]
               : hs        ? __ldg(hs + h)
               : is_v      ? p.w.v_scale
                           : p.w.k_scale;
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const bool is_v = p0 + u >= tensor;
      const int h = (p0 + u - (is_v ? tensor : 0)) * kRows + sub;
      if (p0 + u >= last || h >= hk) continue;
      void* dst = const_cast<void*>(is_v ? p.w.value : p.w.key);
      const int64_t to = t * p.w.src_stride_t + h * p.w.src_stride_h;
      if (type == kBF16 && kJoined) {  // as they are: a conversion would change a NaN's bits
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + to + c0) = make_uint4(a[u].x, a[u].y, b[u].x, b[u].y);
        continue;
      }
      float x[8];
      if (type == kE2M1) {
        e2m1::widen4(a[u].x, x);
        e2m1::widen4(b[u].x, x + 4);
        const float g = __fmul_rn(e2m1::scale1(a[u].y), s[u]), e = __fmul_rn(e2m1::scale1(b[u].y), s[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], i < 4 ? g : e);
      } else if (type == kF32) {
        Chunk<F32>::expand(a[u], x);
        Chunk<F32>::expand(b[u], x + 4);
      } else if (type == kBF16) {
        Chunk<BF16>::expand(make_uint4(a[u].x, a[u].y, b[u].x, b[u].y), x);
      } else {
        if (type == kE4M3) {
          e4m3x4_to_f32x4(a[u].x, x);
          e4m3x4_to_f32x4(b[u].x, x + 4);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)  // (2^23 + code + 128 in the low byte, exact)
            x[i] = __uint_as_float(__byte_perm((i < 4 ? a[u].x : b[u].x) ^ 0x80808080u, 0x4b000000u, 0x7650 + (i & 3))) -
                   8388736.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= s[u];
      }
      store_row<Dst>(dst, to, c0, c1, kJoined, x);
    }
  }
}

// Slices of a token's rows: as many as make a warp for each of the GPU's places (152 SMs x 16),
// down to one pass each; and no slice of more than kFewRows rows, so that many heads do not make
// a warp's work long (a slice computes its token's cosines anew, so fewer are not better).
unsigned slices(int64_t tokens, int rows, int head_dim) {
  const int per_pass = 256 / head_dim, passes = (rows + per_pass - 1) / per_pass;
  int64_t y = (rows + kFewRows - 1) / kFewRows;
  if (tokens * y < 2432) y = (2432 + tokens - 1) / tokens;
  y = y < passes ? y : passes;
  return unsigned(y < 65535 ? y : 65535);
}

template <typename K>
cudaError_t launch(K kern, const TokenParams& p, int rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((p.w.num_tokens + kWarps - 1) / kWarps), slices(p.w.num_tokens, rows, p.w.head_dim));
  cfg.blockDim = dim3(32 * kWarps);
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

template <typename Src, int D, Kind kKind>
cudaError_t launch_rotary(const TokenParams& p, int rows, cudaStream_t stream) {
  if (p.rotary_dim == 0 || p.interleaved) return launch(token_write_kernel<Src, D, kPairs, kKind>, p, rows, stream);
  return p.rotary_dim % 8 == 0 ? launch(token_write_kernel<Src, D, kHalves, kKind>, p, rows, stream)
                               : launch(token_write_kernel<Src, D, kOdd, kKind>, p, rows, stream);
}

template <typename Src, int D>
cudaError_t launch_write(const TokenParams& p, cudaStream_t stream) {
  const int rows = p.num_heads + 2 * p.w.num_kv_heads;
  if (p.num_heads == 0 && p.rotary_dim == 0 && p.w.cache_dtype == kI8)
    return launch(token_quantize_kernel<Src, D>, p, rows, stream);
  if (p.num_heads == 0 && p.rotary_dim == 0 && p.w.cache_dtype == kE2M1)
    return launch(token_four_kernel<Src, D>, p, (rows + 1) / 2, stream);  // (twice the rows a pass)
  if (p.w.cache_dtype == kE2M1) return launch_rotary<Src, D, kFour>(p, rows, stream);
  return p.num_axes ? launch_rotary<Src, D, kAxes>(p, rows, stream) : launch_rotary<Src, D, kPlain>(p, rows, stream);
}

template <typename Dst, int D>
cudaError_t launch_read(const TokenParams& p, cudaStream_t stream) {
  const int rows = 2 * p.w.num_kv_heads;
  switch (p.w.cache_dtype) {
    case kF32: return launch(token_read_kernel<Dst, D, kF32>, p, rows, stream);
    case kBF16: return launch(token_read_kernel<Dst, D, kBF16>, p, rows, stream);
    case kE4M3: return launch(token_read_kernel<Dst, D, kE4M3>, p, rows, stream);
    case kE2M1: return launch(token_read_kernel<Dst, D, kE2M1>, p, rows, stream);
    default: return launch(token_read_kernel<Dst, D, kI8>, p, rows, stream);
  }
}

}  // namespace

cudaError_t launch_token_write(const TokenParams& p, cudaStream_t stream) {
  if (p.w.src_dtype == kBF16)
    return p.w.head_dim == 128 ? launch_write<BF16, 128>(p, stream) : launch_write<BF16, 64>(p, stream);
  return p.w.head_dim == 128 ? launch_write<F32, 128>(p, stream) : launch_write<F32, 64>(p, stream);
}

cudaError_t launch_token_read(const TokenParams& p, cudaStream_t stream) {
  if (p.w.src_dtype == kBF16)
    return p.w.head_dim == 128 ? launch_read<BF16, 128>(p, stream) : launch_read<BF16, 64>(p, stream);
  return p.w.head_dim == 128 ? launch_read<F32, 128>(p, stream) : launch_read<F32, 64>(p, stream);
}

}  // namespace pkv
