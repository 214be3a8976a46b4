// token_api.cu — the C ABI's calls around a step's new tokens (declared in
// include/pkv.h): rotary positions with the cache write, the token-scaled 8-bit cache
// (write, read back, decode) and attention of drafted trees.  Argument checks and kernel
// selection only.
#include <cmath>

#include "pkv_host.h"
#include "token_internal.h"

namespace pkv {
namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

pkv_status check_scales_of(const pkv_tensor* t, const char* name, const pkv_tensor* cache) {
  const pkv_status st = check_scales(t, name);
  if (st) return st;
  for (int i = 0; i < 3; ++i)
    if (t->shape[i] != cache->shape[i])
      return fail(PKV_ERR_INVALID_ARG, "%s must be [num_blocks, num_kv_heads, block_size]", name);
  return PKV_OK;
}

// The caches with, for PKV_I8 ones, their scale arrays.
pkv_status check_caches(const pkv_tensor* kc, const pkv_tensor* vc, const pkv_tensor* ks, const pkv_tensor* vs) {
  pkv_status st;
  if ((st = check_cache(kc, "key_cache", true)) || (st = check_cache(vc, "value_cache", true))) return st;
  if (!same_layout(kc, vc))
    return fail(PKV_ERR_INVALID_ARG, "key_cache and value_cache must share dtype, shape and strides");
  if (!supported_head_dim(kc->shape[3]))
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %lld (supported: 64, 128)", (long long)kc->shape[3]);
  if (!supported_block_size(kc->shape[2]))
    return fail(PKV_ERR_UNSUPPORTED, "block_size %lld (supported: 2, 4, 8, 16, 32)", (long long)kc->shape[2]);
  if (kc->dtype != PKV_I8) {
    if (ks || vs) return fail(PKV_ERR_INVALID_ARG, "k_scales and v_scales are for a token-scaled (i8) cache only");
    return PKV_OK;
  }
  if (!ks || !vs) return fail(PKV_ERR_INVALID_ARG, "an i8 cache needs k_scales and v_scales");
  if ((st = check_scales_of(ks, "k_scales", kc)) || (st = check_scales_of(vs, "v_scales", vc))) return st;
  if (!same_layout(ks, vs)) return fail(PKV_ERR_INVALID_ARG, "k_scales and v_scales must share their strides");
  return PKV_OK;
}

pkv_status check_contiguous(const pkv_tensor* t, const char* name) {
  if (t->shape[0] > 1 && t->stride[0] != 1) return fail(PKV_ERR_INVALID_ARG, "%s must be contiguous", name);
  return PKV_OK;
}

pkv_status check_rows16(const pkv_tensor* t, const char* name) {
  const int eb = elt_bytes(t->dtype);
  if (!aligned16(t->data) || (t->stride[0] * eb) % 16 || (t->stride[1] * eb) % 16)
    return fail(PKV_ERR_INVALID_ARG, "%s: base pointer and strides must be multiples of 16 bytes", name);
  return PKV_OK;
}

// key / value [T, Hk, D] against the caches and the slots; fills the common parameters.
pkv_status token_prepare(const pkv_tensor* key, const pkv_tensor* value, const pkv_tensor* kc, const pkv_tensor* vc,
                         const pkv_tensor* ks, const pkv_tensor* vs, const pkv_tensor* slots, TokenParams* pp) {
  pkv_status st;
  if ((st = check_basic(key, "key", 3)) || (st = check_basic(value, "value", 3)) ||
      (st = check_caches(kc, vc, ks, vs)) || (st = check_basic(slots, "slot_mapping", 1)))
    return st;
  if ((st = check_dtype(key, "key", PKV_F32, PKV_BF16)) || (st = check_dtype(slots, "slot_mapping", PKV_I64)))
    return st;
  if (!same_layout(key, value)) return fail(PKV_ERR_INVALID_ARG, "key and value must share dtype, shape and strides");
  const int64_t T = key->shape[0], Hk = key->shape[1], D = key->shape[2];
  if (kc->shape[1] != Hk || kc->shape[3] != D)
    return fail(PKV_ERR_INVALID_ARG, "key [T, %lld, %lld] does not match the cache's [.., %lld, .., %lld]",
                (long long)Hk, (long long)D, (long long)kc->shape[1], (long long)kc->shape[3]);
  if (slots->shape[0] != T) return fail(PKV_ERR_INVALID_ARG, "slot_mapping must be [num_tokens]");
  if ((st = check_contiguous(slots, "slot_mapping")) || (st = check_rows16(key, "key")) ||
      (st = check_rows16(value, "value")))
    return st;
  if (T > 0x7fffffff || Hk > 65535) return fail(PKV_ERR_UNSUPPORTED, "too many tokens or heads in one call");
  TokenParams& p = *pp;
  p = TokenParams{};
  p.w.key = key->data;
  p.w.value = value->data;
  p.w.src_stride_t = key->stride[0];
  p.w.src_stride_h = key->stride[1];
  p.w.src_dtype = key->dtype;
  p.w.key_cache = kc->data;
  p.w.value_cache = vc->data;
  p.w.cs_block = kc->stride[0];
  p.w.cs_head = kc->stride[1];
  p.w.cache_dtype = kc->dtype;
  p.w.k_scale = kc->scale;
  p.w.v_scale = vc->scale;
  p.w.k_head_scales = kc->head_scales;
  p.w.v_head_scales = vc->head_scales;
  p.w.slot_mapping = static_cast<const int64_t*>(slots->data);
  p.w.num_tokens = T;
  p.w.num_kv_heads = int(Hk);
  p.w.head_dim = int(D);
  p.w.block_size = int(kc->shape[2]);
  p.w.num_blocks = kc->shape[0];
  if (ks) {
    p.k_token_scales = static_cast<float*>(ks->data);
    p.v_token_scales = static_cast<float*>(vs->data);
    p.ts_block = ks->stride[0];
    p.ts_head = ks->stride[1];
  }
  return PKV_OK;
}

// Descriptors and sizes of the attention calls; fills the parameters.  `qsl` and `mask`
// are null for decode.
pkv_status tree_prepare(const pkv_tensor* out, const pkv_tensor* query, const pkv_tensor* kc, const pkv_tensor* vc,
                        const pkv_tensor* ks, const pkv_tensor* vs, const pkv_tensor* tables, const pkv_tensor* lens,
                        const pkv_tensor* qsl, const pkv_tensor* mask, int32_t num_kv_heads, float scale,
                        int32_t block_size, int32_t max_blocks, TreeParams* pp) {
  pkv_status st;
  if ((st = check_basic(out, "out", 3)) || (st = check_basic(query, "query", 3)) ||
      (st = check_caches(kc, vc, ks, vs)) || (st = check_basic(tables, "block_tables", 2)) ||
      (st = check_basic(lens, "context_lens", 1)))
    return st;
  if ((st = check_dtype(query, "query", PKV_F32, PKV_BF16)) ||
      (st = check_dtype(tables, "block_tables", PKV_I32)) || (st = check_dtype(lens, "context_lens", PKV_I32)))
    return st;
  if (out->dtype != query->dtype) return fail(PKV_ERR_INVALID_ARG, "out must have the query's dtype");
  const int64_t T = query->shape[0], Hq = query->shape[1], D = query->shape[2], S = tables->shape[0];
  if (out->shape[0] != T || out->shape[1] != Hq || out->shape[2] != D)
    return fail(PKV_ERR_INVALID_ARG, "out shape must equal query shape [%lld, %lld, %lld]", (long long)T,
                (long long)Hq, (long long)D);
  if (num_kv_heads <= 0 || kc->shape[1] != num_kv_heads)
    return fail(PKV_ERR_INVALID_ARG, "num_kv_heads (%d) must equal key_cache.shape[1] (%lld)", num_kv_heads,
                (long long)kc->shape[1]);
  if (Hq % num_kv_heads)
    return fail(PKV_ERR_INVALID_ARG, "num_heads (%lld) must be a multiple of num_kv_heads (%d)", (long long)Hq,
                num_kv_heads);
  if (kc->shape[2] != block_size || kc->shape[3] != D)
    return fail(PKV_ERR_INVALID_ARG, "block_size / head_dim must match the cache");
  if (tables->shape[1] != max_blocks || max_blocks < 1)
    return fail(PKV_ERR_INVALID_ARG, "block_tables must be [num_seqs, max_blocks_per_seq]");
  if (lens->shape[0] != S || (st = check_contiguous(lens, "context_lens")))
    return fail(PKV_ERR_INVALID_ARG, "context_lens must be a contiguous [num_seqs]");
  if (qsl) {
    if ((st = check_basic(qsl, "query_start_loc", 1)) || (st = check_dtype(qsl, "query_start_loc", PKV_I32)) ||
        (st = check_basic(mask, "tree_mask", 2)) || (st = check_dtype(mask, "tree_mask", PKV_I64)))
      return st;
    if (qsl->shape[0] != S + 1 || check_contiguous(qsl, "query_start_loc"))
      return fail(PKV_ERR_INVALID_ARG, "query_start_loc must be a contiguous [num_seqs + 1]");
    if (mask->shape[0] != T || mask->shape[1] < 1 || mask->shape[1] > 16)
      return fail(PKV_ERR_INVALID_ARG, "tree_mask must be [num_tokens, 1 to 16 words]");
    if (reinterpret_cast<uintptr_t>(mask->data) & 7) return fail(PKV_ERR_INVALID_ARG, "tree_mask must be 8-byte aligned");
  } else if (T != S) {
    return fail(PKV_ERR_INVALID_ARG, "block_tables must be [num_seqs, max_blocks_per_seq], one query per sequence");
  }
  if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "scale must be finite");
  if (int64_t(max_blocks) * block_size > (int64_t(1) << 30)) return fail(PKV_ERR_UNSUPPORTED, "max context above 2^30 tokens");
  if (T > (1 << 28) || S > 65535 || Hq > 65535)
    return fail(PKV_ERR_UNSUPPORTED, "num_seqs and num_heads must be <= 65535, num_tokens <= 2^28");
  if (kc->shape[0] < 1) return fail(PKV_ERR_INVALID_ARG, "the cache holds no block");
  TreeParams& p = *pp;
  p = TreeParams{};
  p.out = out->data;
  p.query = query->data;
  p.q_dtype = query->dtype;
  p.out_stride_t = out->stride[0];
  p.out_stride_h = out->stride[1];
  p.q_stride_t = query->stride[0];
  p.q_stride_h = query->stride[1];
  p.key_cache = kc->data;
  p.value_cache = vc->data;
  p.kv_dtype = kc->dtype;
  p.cs_block = kc->stride[0];
  p.cs_head = kc->stride[1];
  if (ks) {
    p.k_token_scales = static_cast<const float*>(ks->data);
    p.v_token_scales = static_cast<const float*>(vs->data);
    p.ts_block = ks->stride[0];
    p.ts_head = ks->stride[1];
  }
  const bool fp8 = kc->dtype == PKV_FP8_E4M3;
  p.k_head_scales = fp8 ? kc->head_scales : nullptr;
  p.v_head_scales = fp8 ? vc->head_scales : nullptr;
  p.block_tables = static_cast<const int32_t*>(tables->data);
  p.bt_stride = tables->stride[0];
  p.context_lens = static_cast<const int32_t*>(lens->data);
  if (qsl) {
    p.query_start_loc = static_cast<const int32_t*>(qsl->data);
    p.tree_mask = static_cast<const int64_t*>(mask->data);
    p.mask_stride = mask->stride[0];
    p.mask_words = int(mask->shape[1]);
  }
  p.num_seqs = int(S);
  p.num_tokens = int(T);
  p.num_heads = int(Hq);
  p.num_kv_heads = num_kv_heads;
  p.group = int(Hq / num_kv_heads);
  p.head_dim = int(D);
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks;
  p.num_blocks = kc->shape[0];
  p.qk_scale_log2 = float(double(scale) * 1.4426950408889634 * double(fp8 && !p.k_head_scales ? kc->scale : 1.f));
  p.v_scale = fp8 && !p.v_head_scales ? vc->scale : 1.f;
  return PKV_OK;
}

// f radians as a part of a turn in units of 2^-96, rounded to nearest: *high 2^32 + *low.  f is
// taken as the number that it is, m 2^e, and the turn from a product of whole numbers, so that
// nothing is lost but the last bit: at position p the angle is off by at most p 2^-97 turns.
// |f| <= 2^64, so that the 256 bits of 1 / 2 pi below are enough.
void radians_to_turn(double f, uint64_t* high, uint32_t* low) {
  static const uint64_t kInverse[4] = {0x7f9458eaf7aef158ull, 0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull,
                                       0x28be60db9391054aull};  // floor(2^256 / 2 pi), lowest first
  int e;
  const uint64_t m = uint64_t(std::ldexp(std::frexp(std::fabs(f), &e), 53));  // (exact)
  uint64_t x[7] = {0, 0, 0, 0, 0, 0, 0}, carry = 0;  // m / 2 pi, in units of 2^-256
  for (int i = 0; i < 4; ++i) {
    const unsigned __int128 y = static_cast<unsigned __int128>(m) * kInverse[i] + carry;
    x[i] = uint64_t(y);
    carry = uint64_t(y >> 64);
  }
  x[4] = carry;
  const int shift = 160 - (e - 53);  // of units of 2^-256 to those of 2^-96, for m 2^(e - 53)
  if (shift > 320) {  // (less than half a unit)
    *high = 0;
    *low = 0;
    return;
  }
  auto bits = [&](int at) {  // 64 of them from bit `at` on
    const int w = at >> 6, o = at & 63;
    return o ? x[w] >> o | x[w + 1] << (64 - o) : x[w];
  };
  unsigned __int128 n = static_cast<unsigned __int128>(bits(shift)) |
                        static_cast<unsigned __int128>(shift + 64 < 384 ? bits(shift + 64) : 0) << 64;
  n += bits(shift - 1) & 1;
  if (f < 0) n = -n;
  *high = uint64_t(n >> 32);
  *low = uint32_t(n);
}

// Blocks of a tensor-core kernel.
int tree_grid(int num_sms, int per_sm) {
  return per_sm * (num_sms < int(TreeSplit::kMaxSms) ? num_sms : int(TreeSplit::kMaxSms));
}

pkv_status tree_launch(TreeParams& p, cudaStream_t stream, const char* what) {
  if (dry_run() || p.num_seqs == 0 || p.num_tokens == 0 || p.num_heads == 0) return PKV_OK;
  DeviceState* s;
  pkv_status st = device_state(&s);
  if (st) return st;
  p.err = s->err;
  if (!tree_tensor_supported(p)) return finish_call(s, launch_tree_core(p, stream), stream, what);
  const int grid = tree_grid(s->num_sms, decode_i8_supported(p) ? decode_i8_blocks_per_sm(p.group) : 1);
  const int rows = tree_part_rows(p.num_tokens, p.group, !p.query_start_loc, p.kv_dtype == kI8);
  std::unique_lock<std::mutex> use(s->ws_use);
  if ((st = ensure_workspace(s, tree_workspace(grid, rows, p.head_dim), stream))) return st;
  return finish_call(s, launch_tree_tensor(p, grid, rows, s->ws, stream), stream, what);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_rotary_init(pkv_rotary* rotary, int32_t rotary_dim, int32_t interleaved, double base, int32_t scaling,
                           double factor, int64_t original) {
  if (!rotary) return fail(PKV_ERR_INVALID_ARG, "null rotary pointer");
  if (rotary_dim < 0 || rotary_dim > 128 || rotary_dim % 2)
    return fail(PKV_ERR_INVALID_ARG, "rotary_dim must be even, 0 to 128");
  if (interleaved != 0 && interleaved != 1) return fail(PKV_ERR_INVALID_ARG, "interleaved is 0 or 1");
  if (!(std::isfinite(base) && base > 1.0)) return fail(PKV_ERR_INVALID_ARG, "base must be finite and above 1");
  if (scaling < PKV_ROTARY_NONE || scaling > PKV_ROTARY_RAMP)
    return fail(PKV_ERR_INVALID_ARG, "unknown rotary scaling %d", scaling);
  if (scaling != PKV_ROTARY_NONE && !(std::isfinite(factor) && factor >= 1.0))
    return fail(PKV_ERR_INVALID_ARG, "the scaling factor must be finite and >= 1");
  if ((scaling == PKV_ROTARY_BANDS || scaling == PKV_ROTARY_RAMP) && original < 1)
    return fail(PKV_ERR_INVALID_ARG, "this scaling needs the original context length");
  *rotary = pkv_rotary{};
  rotary->rotary_dim = rotary_dim;
  rotary->interleaved = interleaved;
  rotary->magnitude = scaling == PKV_ROTARY_RAMP ? 0.1 * std::log(factor) + 1.0 : 1.0;
  const double d = rotary_dim;
  if (scaling == PKV_ROTARY_BASE && rotary_dim > 2) base *= std::pow(factor, d / (d - 2.0));
  // (RAMP) the index, not whole, of the pair that makes r turns over the original context
  auto index_of = [&](double r) { return d * std::log(double(original) / (r * kTwoPi)) / (2.0 * std::log(base)); };
  double first = 0.0, last = 0.0;
  if (scaling == PKV_ROTARY_RAMP) {
    first = std::fmax(std::floor(index_of(32.0)), 0.0);
    last = std::fmin(std::ceil(index_of(1.0)), d - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / d);
    double keep = 1.0;  // the unscaled share
    if (scaling == PKV_ROTARY_LINEAR) keep = 0.0;
    if (scaling == PKV_ROTARY_BANDS) keep = std::fmin(1.0, std::fmax(0.0, (double(original) * f / kTwoPi - 1.0) / 3.0));
    if (scaling == PKV_ROTARY_RAMP)
      keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - first) / std::fmax(last - first, 1e-3)));
    const bool scaled = scaling != PKV_ROTARY_NONE && scaling != PKV_ROTARY_BASE;
    rotary->frequency[i] = scaled ? f * keep + f / factor * (1.0 - keep) : f;
  }
  return PKV_OK;
}

pkv_status pkv_rotary_and_cache(const pkv_tensor* query_out, const pkv_tensor* query, const pkv_tensor* key,
                                const pkv_tensor* value, const pkv_tensor* positions, const pkv_tensor* key_cache,
                                const pkv_tensor* value_cache, const pkv_tensor* k_scales, const pkv_tensor* v_scales,
                                const pkv_tensor* slot_mapping, const pkv_rotary* rotary, pkv_stream stream) {
  TokenParams p;
  pkv_status st = token_prepare(key, value, key_cache, value_cache, k_scales, v_scales, slot_mapping, &p);
  if (st) return st;
  if ((st = check_basic(query, "query", 3)) || (st = check_basic(query_out, "query_out", 3)) ||
      (st = check_basic(positions, "positions", 1)) ||
      (st = check_dtype(positions, "positions", PKV_I32, PKV_I64)) || (st = check_contiguous(positions, "positions")))
    return st;
  const int64_t T = key->shape[0], D = key->shape[2];
  if (query->dtype != key->dtype || query_out->dtype != key->dtype)
    return fail(PKV_ERR_INVALID_ARG, "query, query_out, key and value must share a dtype");
  if (query->shape[0] != T || query->shape[2] != D)
    return fail(PKV_ERR_INVALID_ARG, "query must be [num_tokens=%lld, num_heads, head_dim=%lld]", (long long)T,
                (long long)D);
  for (int i = 0; i < 3; ++i)
    if (query_out->shape[i] != query->shape[i]) return fail(PKV_ERR_INVALID_ARG, "query_out shape must equal query shape");
  if ((st = check_rows16(query, "query")) || (st = check_rows16(query_out, "query_out"))) return st;
  if (query_out->data == query->data &&
      (query_out->stride[0] != query->stride[0] || query_out->stride[1] != query->stride[1]))
    return fail(PKV_ERR_INVALID_ARG, "query_out in place of query must have its strides");
  if (positions->shape[0] != T) return fail(PKV_ERR_INVALID_ARG, "positions must be [num_tokens]");
  const int c = key_cache->dtype;
  if (c != key->dtype && c != PKV_FP8_E4M3 && c != PKV_I8)
    return fail(PKV_ERR_UNSUPPORTED, "writing %s tokens into a %s cache", dtype_name(key->dtype), dtype_name(c));
  if (!rotary) return fail(PKV_ERR_INVALID_ARG, "null rotary pointer");
  if (rotary->rotary_dim < 0 || rotary->rotary_dim % 2 || rotary->rotary_dim > D)
    return fail(PKV_ERR_INVALID_ARG, "rotary_dim (%d) must be even, 0 to head_dim (%lld)", rotary->rotary_dim, (long long)D);
  if (rotary->interleaved != 0 && rotary->interleaved != 1) return fail(PKV_ERR_INVALID_ARG, "interleaved is 0 or 1");
  if (!std::isfinite(float(rotary->magnitude)))
    return fail(PKV_ERR_INVALID_ARG, "the rotary magnitude must be finite in binary32");
  if (query->shape[1] > 65535) return fail(PKV_ERR_UNSUPPORTED, "too many heads");
  p.query = query->data;
  p.query_out = query_out->data;
  p.q_stride_t = query->stride[0];
  p.q_stride_h = query->stride[1];
  p.qo_stride_t = query_out->stride[0];
  p.qo_stride_h = query_out->stride[1];
  p.num_heads = int(query->shape[1]);
  p.positions = positions->data;
  p.positions64 = positions->dtype == PKV_I64;
  p.rotary_dim = rotary->rotary_dim;
  p.interleaved = rotary->interleaved != 0;
  p.magnitude = float(rotary->magnitude);
  for (int i = 0; i < rotary->rotary_dim / 2; ++i) {
    const double f = rotary->frequency[i];
    if (!(std::fabs(f) <= 0x1p64))
      return fail(PKV_ERR_INVALID_ARG, "rotary frequency %d is not a number of at most 2^64 in magnitude", i);
    radians_to_turn(f, &p.turns[i], &p.turns_low[i]);
  }
  if (dry_run() || T == 0 || (p.num_heads == 0 && p.w.num_kv_heads == 0)) return PKV_OK;
  DeviceState* s;
  if ((st = device_state(&s))) return st;
  p.w.err = s->err;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return finish_call(s, launch_token_write(p, cs), cs, "rotary_and_cache");
}

pkv_status pkv_quantize_and_cache(const pkv_tensor* key, const pkv_tensor* value, const pkv_tensor* key_cache,
                                  const pkv_tensor* value_cache, const pkv_tensor* k_scales, const pkv_tensor* v_scales,
                                  const pkv_tensor* slot_mapping, pkv_stream stream) {
  TokenParams p;
  pkv_status st = token_prepare(key, value, key_cache, value_cache, k_scales, v_scales, slot_mapping, &p);
  if (st) return st;
  if (key_cache->dtype != PKV_I8)
    return fail(PKV_ERR_UNSUPPORTED, "quantize_and_cache writes i8 caches (got %s)", dtype_name(key_cache->dtype));
  if (dry_run() || p.w.num_tokens == 0 || p.w.num_kv_heads == 0) return PKV_OK;
  DeviceState* s;
  if ((st = device_state(&s))) return st;
  p.w.err = s->err;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return finish_call(s, launch_token_write(p, cs), cs, "quantize_and_cache");
}

pkv_status pkv_read_cache(const pkv_tensor* key, const pkv_tensor* value, const pkv_tensor* key_cache,
                          const pkv_tensor* value_cache, const pkv_tensor* k_scales, const pkv_tensor* v_scales,
                          const pkv_tensor* slot_mapping, pkv_stream stream) {
  TokenParams p;
  pkv_status st = token_prepare(key, value, key_cache, value_cache, k_scales, v_scales, slot_mapping, &p);
  if (st) return st;
  if (dry_run() || p.w.num_tokens == 0 || p.w.num_kv_heads == 0) return PKV_OK;
  DeviceState* s;
  if ((st = device_state(&s))) return st;
  p.w.err = s->err;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return finish_call(s, launch_token_read(p, cs), cs, "read_cache");
}

pkv_status pkv_paged_attention_decode_quantized(const pkv_tensor* out, const pkv_tensor* query,
                                                const pkv_tensor* key_cache, const pkv_tensor* value_cache,
                                                const pkv_tensor* k_scales, const pkv_tensor* v_scales,
                                                const pkv_tensor* block_tables, const pkv_tensor* context_lens,
                                                int32_t num_kv_heads, float scale, int32_t block_size,
                                                int32_t max_blocks_per_seq, int32_t sliding_window, pkv_stream stream) {
  TreeParams p;
  pkv_status st = tree_prepare(out, query, key_cache, value_cache, k_scales, v_scales, block_tables, context_lens,
                               nullptr, nullptr, num_kv_heads, scale, block_size, max_blocks_per_seq, &p);
  if (st) return st;
  if (key_cache->dtype != PKV_I8)
    return fail(PKV_ERR_UNSUPPORTED, "decode_quantized reads i8 caches (got %s)", dtype_name(key_cache->dtype));
  if (sliding_window < 0) return fail(PKV_ERR_INVALID_ARG, "sliding_window must be >= 0 (0: no window)");
  p.sliding_window = sliding_window;
  return tree_launch(p, static_cast<cudaStream_t>(stream), "paged_attention_decode_quantized");
}

pkv_status pkv_paged_attention_tree(const pkv_tensor* out, const pkv_tensor* query, const pkv_tensor* key_cache,
                                    const pkv_tensor* value_cache, const pkv_tensor* k_scales,
                                    const pkv_tensor* v_scales, const pkv_tensor* block_tables,
                                    const pkv_tensor* context_lens, const pkv_tensor* query_start_loc,
                                    const pkv_tensor* tree_mask, int32_t num_kv_heads, float scale, int32_t block_size,
                                    int32_t max_blocks_per_seq, pkv_stream stream) {
  if (!query_start_loc) return fail(PKV_ERR_INVALID_ARG, "query_start_loc: null descriptor");
  TreeParams p;
  const pkv_status st = tree_prepare(out, query, key_cache, value_cache, k_scales, v_scales, block_tables, context_lens,
                                     query_start_loc, tree_mask, num_kv_heads, scale, block_size, max_blocks_per_seq, &p);
  if (st) return st;
  return tree_launch(p, static_cast<cudaStream_t>(stream), "paged_attention_tree");
}

int64_t pkv_tree_workspace_bytes(int32_t num_seqs, int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                                 int32_t head_dim) {
  if (num_seqs <= 0 || num_tokens <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      num_heads % num_kv_heads)
    return 0;
  const int group = num_heads / num_kv_heads;
  if (group > 128) return 0;
  int num_sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    num_sms = int(TreeSplit::kMaxSms);
  const size_t tree = tree_workspace(tree_grid(num_sms, 1), tree_part_rows(num_tokens, group, false, false), head_dim);
  const size_t decode = tree_workspace(tree_grid(num_sms, decode_i8_blocks_per_sm(group)),
                                       tree_part_rows(num_tokens, group, true, false), head_dim);
  return int64_t(tree > decode || group > 16 ? tree : decode);
}

}  // extern "C"
