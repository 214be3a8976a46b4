"""ctypes binding of libpkv (include/pkv.h).

Argument marshalling only: each function turns torch tensors into pkv_tensor
descriptors (device pointer, dtype, shape, strides, fp8 scale), passes the current
CUDA stream, and raises :class:`PkvError` on a non-OK status.  Every step of the work
runs in the library's CUDA kernels; if the library is not built this module raises
instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libpkv.so")

PKV_OK = 0
STATUS_NAMES = {0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_UNSUPPORTED", 3: "PKV_ERR_CUDA",
                4: "PKV_ERR_DEVICE_CHECK"}
DEVERR = {"table_entry": 0x1, "slot": 0x2, "copy_pair": 0x4, "context_len": 0x8, "timeout": 0x10,
          "copy_overlap": 0x20, "keep": 0x40}
OPTIONS = {"partition_tokens": 0, "debug_sync": 1, "dry_run": 2, "decode_kernel": 3,
           "dynamic_share": 4, "dynamic_chunk": 5, "fused_append": 6,
           "prefill_kernel": 7}
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2, torch.int32: 3, torch.int64: 4,
           torch.int8: 5, torch.uint8: 6}
if hasattr(torch, "float4_e2m1fn_x2"):
    _DTYPES[torch.float4_e2m1fn_x2] = 6  # a 4-bit cache's bytes, as torch.uint8
ROTARY_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


class PkvTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4), ("scale", ctypes.c_float),
                ("head_scales", ctypes.c_void_p)]


class PkvRotary(ctypes.Structure):
    """pkv_rotary: how rotary_and_cache turns queries and keys (see :func:`rotary`)."""
    axes: "Optional[PkvRotaryAxes]" = None  # with several position axes
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("magnitude", ctypes.c_double),
                ("frequency", ctypes.c_double * 64)]


class PkvRotaryAxes(ctypes.Structure):
    """pkv_rotary_axes: which position axis turns each pair."""
    _fields_ = [("num_axes", ctypes.c_int32), ("axis", ctypes.c_int32 * 64)]


_lock = threading.Lock()
_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libpkv.so (built in-tree by paged_kv_cache_90_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with `python -m paged_kv_cache_90_gb300.build` "
                               "(or __graft_entry__.build()); there is no fallback path")
        lib = ctypes.CDLL(p)
        d = ctypes.POINTER(PkvTensor)
        i32, i64, f32, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
        lib.pkv_paged_attention_decode.argtypes = [d, d, d, d, d, d, i32, f32, i32, i32, vp]
        lib.pkv_reshape_and_cache.argtypes = [d, d, d, d, d, vp]
        lib.pkv_copy_blocks.argtypes = [d, d, vp]
        lib.pkv_paged_attention_decode_noalloc.argtypes = [d, d, d, d, d, d, i32, f32, i32, i32, vp]
        lib.pkv_decode_step.argtypes = [d, d, d, d, d, d, d, d, d, i32, f32, i32, i32, i32, vp]
        lib.pkv_reshape_and_cache_amax.argtypes = [d, d, d, d, d, vp, vp, vp]
        lib.pkv_paged_attention_prefill.argtypes = [d, d, d, d, d, d, d, i32, f32, i32, i32, vp]
        lib.pkv_decode_append.argtypes = [d, d, d, d, d, d, d, d, d, i32, f32, i32, i32, i32, vp]
        lib.pkv_paged_attention_decode_window.argtypes = [d, d, d, d, d, d, i32, f32, i32, i32, i32, vp]
        lib.pkv_rotary_init.argtypes = [ctypes.POINTER(PkvRotary), i32, i32, ctypes.c_double, i32, ctypes.c_double,
                                        i64]
        lib.pkv_rotary_and_cache.argtypes = [d] * 10 + [ctypes.POINTER(PkvRotary), vp]
        lib.pkv_rotary_axes_and_cache.argtypes = [d] * 10 + [ctypes.POINTER(PkvRotary),
                                                             ctypes.POINTER(PkvRotaryAxes), vp]
        lib.pkv_copy_cache_blocks.argtypes = [ctypes.POINTER(d), i32, d, vp]
        lib.pkv_keep_tokens.argtypes = [ctypes.POINTER(d), i32] + [d] * 6 + [i32, i32, vp]
        lib.pkv_quantize_and_cache.argtypes = [d] * 7 + [vp]
        lib.pkv_read_cache.argtypes = [d] * 7 + [vp]
        lib.pkv_paged_attention_decode_quantized.argtypes = [d] * 8 + [i32, f32, i32, i32, i32, vp]
        lib.pkv_paged_attention_tree.argtypes = [d] * 10 + [i32, f32, i32, i32, vp]
        lib.pkv_tree_workspace_bytes.restype = i64
        lib.pkv_tree_workspace_bytes.argtypes = [i32] * 5
        lib.pkv_noalloc_scratch_bytes.restype = i64
        lib.pkv_noalloc_scratch_bytes.argtypes = []
        for fn in ("pkv_paged_attention_decode", "pkv_paged_attention_decode_noalloc",
                   "pkv_reshape_and_cache", "pkv_decode_step", "pkv_copy_blocks",
                   "pkv_paged_attention_decode_window", "pkv_reshape_and_cache_amax",
                   "pkv_paged_attention_prefill", "pkv_decode_append", "pkv_rotary_init",
                   "pkv_rotary_and_cache", "pkv_quantize_and_cache", "pkv_read_cache",
                   "pkv_paged_attention_decode_quantized", "pkv_paged_attention_tree",
                   "pkv_rotary_axes_and_cache", "pkv_copy_cache_blocks", "pkv_keep_tokens",
                   "pkv_set_option", "pkv_reserve_workspace", "pkv_read_device_errors"):
            getattr(lib, fn).restype = ctypes.c_int
        lib.pkv_last_error.restype = ctypes.c_char_p
        lib.pkv_last_error.argtypes = []
        lib.pkv_abi_version.restype = i32
        lib.pkv_set_option.argtypes = [i32, i64]
        lib.pkv_get_option.restype = i64
        lib.pkv_get_option.argtypes = [i32]
        lib.pkv_reserve_workspace.argtypes = [i64]
        lib.pkv_decode_workspace_bytes.restype = i64
        lib.pkv_decode_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.pkv_read_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
        lib.pkv_launch_count.restype = ctypes.c_uint64
        lib.pkv_launch_count.argtypes = []
        _lib = lib
        return lib


def _check(status: int) -> None:
    if status != PKV_OK:
        msg = load_library().pkv_last_error()
        raise PkvError(status, msg.decode() if msg else "")


def describe(t: torch.Tensor, scale: float = 1.0, head_scales: Optional[torch.Tensor] = None) -> PkvTensor:
    """pkv_tensor descriptor of a tensor (pointer, dtype code, shape, strides); an 8-bit or
    4-bit cache may carry one scale per KV head (a float32 tensor on the cache's device)."""
    if t.dim() > 4 or t.dim() < 1:
        raise ValueError("descriptors cover 1 to 4 dimensions")
    if t.dtype not in _DTYPES:
        raise TypeError(f"dtype {t.dtype} has no pkv code")
    d = PkvTensor()
    d.data = t.data_ptr() if t.numel() else None
    d.dtype = _DTYPES[t.dtype]
    d.ndim = t.dim()
    for i in range(4):
        d.shape[i] = t.shape[i] if i < t.dim() else 1
        d.stride[i] = t.stride(i) if i < t.dim() else 1
    d.scale = float(scale)
    if head_scales is not None:
        if head_scales.dtype != torch.float32 or not head_scales.is_contiguous() or head_scales.device != t.device:
            raise ValueError("head scales must be a contiguous float32 tensor on the cache's device")
        d.head_scales = head_scales.data_ptr()
    return d


# Descriptors the call wrappers pass, by everything a descriptor holds (address, dtype,
# shape, strides, scale, per-head scales): a serving loop passes the same tensors every
# step, and building a descriptor costs several microseconds of Python.  The cached
# objects never leave this module, so nothing mutates them.  A key of four parts is that of
# a tensor without scales, which most are (looking at less halves the cost).
_DESC_CACHE: dict = {}
_DESC_CACHE_MAX = 4096


def _ref(t: torch.Tensor, scale: float = 1.0, head_scales: Optional[torch.Tensor] = None):
    if scale == 1.0 and head_scales is None:
        key = (t.data_ptr(), t.dtype, t.shape, t.stride())
        r = _DESC_CACHE.get(key)
        if r is None:
            if len(_DESC_CACHE) >= _DESC_CACHE_MAX:
                _DESC_CACHE.clear()
            r = _DESC_CACHE[key] = ctypes.byref(describe(t))
        return r
    hs = None if head_scales is None else (head_scales.data_ptr(), head_scales.dtype, head_scales.device,
                                             head_scales.stride())
    key = (t.data_ptr(), t.dtype, t.device, t.shape, t.stride(), float(scale), hs)
    r = _DESC_CACHE.get(key)
    if r is None:
        if len(_DESC_CACHE) >= _DESC_CACHE_MAX:
            _DESC_CACHE.clear()
        r = _DESC_CACHE[key] = ctypes.byref(describe(t, scale, head_scales))
    return r


_have_cuda = False  # (asked until the answer is yes: the question costs microseconds)
# The current stream's handle alone (a Stream object takes 3 us to make, a fifth of a small
# call).  Not a public name of torch's: where it is missing the Stream object is asked.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> ctypes.c_void_p:
    global _have_cuda
    if stream is None:
        if not _have_cuda:
            _have_cuda = torch.cuda.is_available()
            if not _have_cuda:
                return ctypes.c_void_p(0)
        device = torch.cuda.current_device()
        return ctypes.c_void_p(_raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def paged_attention_decode(out, query, key_cache, value_cache, block_tables, context_lens,
                           num_kv_heads: int, scale: float, block_size: int,
                           max_blocks_per_seq: int, k_scale: float = 1.0, v_scale: float = 1.0,
                           stream=None, sliding_window: int = 0, k_head_scales=None,
                           v_head_scales=None) -> torch.Tensor:
    """Single-token decode attention over the paged cache into ``out`` (returned).
    ``sliding_window`` W > 0: each sequence attends to its last W positions only
    (pkv_paged_attention_decode_window).  ``k_head_scales`` / ``v_head_scales``: one
    scale per KV head of an 8-bit cache (device float32), instead of k_scale / v_scale."""
    lib = load_library()
    descs = [_ref(out), _ref(query), _ref(key_cache, k_scale, k_head_scales),
             _ref(value_cache, v_scale, v_head_scales), _ref(block_tables), _ref(context_lens)]
    if sliding_window:
        _check(lib.pkv_paged_attention_decode_window(*descs, int(num_kv_heads), float(scale), int(block_size),
                                                     int(max_blocks_per_seq), int(sliding_window),
                                                     _stream(stream)))
    else:
        _check(lib.pkv_paged_attention_decode(*descs, int(num_kv_heads), float(scale), int(block_size),
                                              int(max_blocks_per_seq), _stream(stream)))
    return out


def decode_step(out, query, key, value, slot_mapping, key_cache, value_cache, block_tables, context_lens,
                num_kv_heads: int, scale: float, block_size: int, max_blocks_per_seq: int,
                k_scale: float = 1.0, v_scale: float = 1.0, stream=None,
                sliding_window: int = 0, k_head_scales=None, v_head_scales=None) -> torch.Tensor:
    """Append the step's new tokens (``key``/``value`` at ``slot_mapping``) to the cache
    and decode into ``out`` (returned): the results of reshape_and_cache followed by
    paged_attention_decode, with the decode's preparation overlapping the write."""
    lib = load_library()
    descs = [_ref(out), _ref(query), _ref(key), _ref(value), _ref(slot_mapping),
             _ref(key_cache, k_scale, k_head_scales), _ref(value_cache, v_scale, v_head_scales),
             _ref(block_tables), _ref(context_lens)]
    _check(lib.pkv_decode_step(*descs, int(num_kv_heads), float(scale),
                               int(block_size), int(max_blocks_per_seq), int(sliding_window), _stream(stream)))
    return out


def prepare_decode_step(out, query, key, value, slot_mapping, key_cache, value_cache, block_tables,
                        context_lens, num_kv_heads: int, scale: float, block_size: int, max_blocks_per_seq: int,
                        k_scale: float = 1.0, v_scale: float = 1.0, stream=None, sliding_window: int = 0,
                        k_head_scales=None, v_head_scales=None):
    """decode_step's arguments marshalled once: the returned callable issues that same
    call (same tensors, same stream, resolved now) each time it is called, with nothing
    rebuilt, for serving loops that reuse their buffers every step.  The tensors must
    stay alive, on the same storage, shapes and strides, while the callable is used (it
    holds references to them).  Each call returns ``out``."""
    lib = load_library()
    keep = (out, query, key, value, slot_mapping, key_cache, value_cache, block_tables, context_lens,
            k_head_scales, v_head_scales)
    descs = [describe(out), describe(query), describe(key), describe(value), describe(slot_mapping),
             describe(key_cache, k_scale, k_head_scales), describe(value_cache, v_scale, v_head_scales),
             describe(block_tables), describe(context_lens)]
    args = tuple(ctypes.byref(d) for d in descs) + (
        ctypes.c_int32(int(num_kv_heads)), ctypes.c_float(float(scale)), ctypes.c_int32(int(block_size)),
        ctypes.c_int32(int(max_blocks_per_seq)), ctypes.c_int32(int(sliding_window)), _stream(stream))
    fn = lib.pkv_decode_step

    def call() -> torch.Tensor:
        _check(fn(*args))
        return out

    call.tensors, call.descriptors = keep, descs  # kept alive with the callable
    return call


def decode_append(out, query, key, value, slot_mapping, key_cache, value_cache, block_tables, context_lens,
                  num_kv_heads: int, scale: float, block_size: int, max_blocks_per_seq: int,
                  k_scale: float = 1.0, v_scale: float = 1.0, stream=None, sliding_window: int = 0,
                  k_head_scales=None, v_head_scales=None) -> torch.Tensor:
    """decode_step for one new token per sequence (token s of ``key`` / ``value`` is
    sequence s's newest, its slot the position context_lens[s] - 1); with the
    ``fused_append`` option at 2 the write runs inside the decode kernel.  Returns
    ``out``."""
    lib = load_library()
    descs = [_ref(out), _ref(query), _ref(key), _ref(value), _ref(slot_mapping),
             _ref(key_cache, k_scale, k_head_scales), _ref(value_cache, v_scale, v_head_scales),
             _ref(block_tables), _ref(context_lens)]
    _check(lib.pkv_decode_append(*descs, int(num_kv_heads), float(scale),
                                 int(block_size), int(max_blocks_per_seq), int(sliding_window), _stream(stream)))
    return out


def paged_attention_prefill(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc,
                            num_kv_heads: int, scale: float, block_size: int, max_blocks_per_seq: int,
                            stream=None) -> torch.Tensor:
    """Causal attention of the packed new tokens of every sequence (rows
    query_start_loc[s] .. query_start_loc[s+1]-1, the last of its context_lens[s]
    cached positions) over the paged cache, into ``out`` (returned)."""
    lib = load_library()
    descs = [_ref(out), _ref(query), _ref(key_cache), _ref(value_cache), _ref(block_tables),
             _ref(context_lens), _ref(query_start_loc)]
    _check(lib.pkv_paged_attention_prefill(*descs, int(num_kv_heads), float(scale),
                                           int(block_size), int(max_blocks_per_seq), _stream(stream)))
    return out


def paged_attention_decode_noalloc(out, query, key_cache, value_cache, block_tables, context_lens,
                                   num_kv_heads: int, scale: float, block_size: int,
                                   max_blocks_per_seq: int, k_scale: float = 1.0,
                                   v_scale: float = 1.0, stream=None) -> torch.Tensor:
    """Decode attention that allocates no device memory: partial results of split
    contexts go to the library's fixed 16 MiB scratch array instead of a workspace
    grown with cudaMalloc (for callers that own all device memory, or must not let
    an allocation synchronise the device).  Calls on one device share that scratch,
    so calls on unordered streams must not overlap."""
    lib = load_library()
    descs = [_ref(out), _ref(query), _ref(key_cache, k_scale),
             _ref(value_cache, v_scale), _ref(block_tables), _ref(context_lens)]
    _check(lib.pkv_paged_attention_decode_noalloc(*descs,
                                                  int(num_kv_heads), float(scale), int(block_size),
                                                  int(max_blocks_per_seq), _stream(stream)))
    return out


def noalloc_scratch_bytes() -> int:
    return int(load_library().pkv_noalloc_scratch_bytes())


def reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, k_scale: float = 1.0,
                      v_scale: float = 1.0, stream=None, k_head_scales=None, v_head_scales=None,
                      k_amax=None, v_amax=None) -> None:
    """Write the new tokens' K/V into their cache slots (in place).  ``k_amax`` /
    ``v_amax`` (device float32 [Hk], starting >= 0) are raised to the largest |x|
    written per KV head (pkv_reshape_and_cache_amax)."""
    lib = load_library()
    descs = [_ref(key), _ref(value), _ref(key_cache, k_scale, k_head_scales),
             _ref(value_cache, v_scale, v_head_scales), _ref(slot_mapping)]
    if k_amax is None and v_amax is None:
        _check(lib.pkv_reshape_and_cache(*descs, _stream(stream)))
        return
    for a in (k_amax, v_amax):
        if a is not None and (a.dtype != torch.float32 or not a.is_contiguous() or a.device != key_cache.device):
            raise ValueError("amax arrays must be contiguous float32 tensors on the cache's device")
    _check(lib.pkv_reshape_and_cache_amax(*descs, None if k_amax is None else ctypes.c_void_p(k_amax.data_ptr()),
                                          None if v_amax is None else ctypes.c_void_p(v_amax.data_ptr()),
                                          _stream(stream)))


def copy_blocks(cache, src_dst_pairs, stream=None) -> None:
    """cache[dst] = cache[src] for every (src, dst) row of ``src_dst_pairs``; ``cache`` may be
    the scale array of an int8 cache or the group scales of a 4-bit one, which are copied like it.
    copy_cache_blocks takes the caches of all layers at once."""
    lib = load_library()
    pairs = src_dst_pairs
    if pairs.numel() == 0:
        pairs = pairs.reshape(0, 2)
    descs = [_ref(cache), _ref(pairs)]
    _check(lib.pkv_copy_blocks(*descs, _stream(stream)))


class CacheList:
    """The caches (and scale arrays) of all layers, marshalled once for the calls that take
    many: see :func:`cache_list`.  Holds references to them."""

    def __init__(self, caches):
        self.caches = tuple(caches)
        if not self.caches:
            raise ValueError("a cache list holds at least one cache")
        if len({c.device for c in self.caches}) != 1:
            raise ValueError("the caches of a list must be on one device")
        self._descs = [describe(c) for c in self.caches]
        self._array = (ctypes.POINTER(PkvTensor) * len(self._descs))(*[ctypes.pointer(x) for x in self._descs])

    def __len__(self) -> int:
        return len(self.caches)


def cache_list(caches) -> CacheList:
    """Made once, passed to every copy_cache_blocks and keep_tokens: caches [num_blocks, Hk,
    block_size, ...] of any dtypes with one num_blocks and block_size, and their scale arrays.  The
    tensors must stay on the same storage, shapes and strides while the list is used."""
    return CacheList(caches)


def copy_cache_blocks(caches, src_dst_pairs, stream=None) -> None:
    """cache[dst] = cache[src] for every (src, dst) row of ``src_dst_pairs`` (int64) in every
    cache of ``caches`` (a :func:`cache_list`, or the tensors), in one launch: a fork's or a
    copy-on-write's private blocks, or the moves that pack a fragmented pool
    (:meth:`block_manager.BlockManager.compact`)."""
    lib = load_library()
    if not isinstance(caches, CacheList):
        caches = CacheList(caches)
    pairs = src_dst_pairs
    if pairs.numel() == 0:
        pairs = pairs.reshape(0, 2)
    _check(lib.pkv_copy_cache_blocks(caches._array, len(caches), _ref(pairs), _stream(stream)))


def keep_tokens(caches, block_tables, context_lens, query_start_loc, keep, keep_counts, block_size: int,
                max_blocks_per_seq: int, new_lens=None, stream=None):
    """Keep the drafted tokens that were accepted, in every cache of ``caches`` (a
    :func:`cache_list`, or the tensors): of sequence s's drafted nodes (the last
    query_start_loc[s+1] - query_start_loc[s] of its context_lens[s] cached tokens) the first
    keep_counts[s] entries of ``keep`` from query_start_loc[s] on, in ascending order, move to the
    positions that follow the context.  ``new_lens`` (int32, returned) receives the lengths."""
    lib = load_library()
    if not isinstance(caches, CacheList):
        caches = CacheList(caches)
    _check(lib.pkv_keep_tokens(caches._array, len(caches), _ref(block_tables), _ref(context_lens),
                               _ref(query_start_loc), _ref(keep), _ref(keep_counts), _opt_ref(new_lens),
                               int(block_size), int(max_blocks_per_seq), _stream(stream)))
    return new_lens


def rotary(rotary_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
           factor: float = 1.0, original_max_position: int = 0, frequencies=None,
           magnitude: Optional[float] = None, axes=None) -> PkvRotary:
    """The rotation that rotary_and_cache applies: made once, passed to every call.  The
    first ``rotary_dim`` columns of a head are rotated, in pairs half of them apart or
    (``interleaved``) next to each other.  ``scaling`` (none, linear, base, bands, ramp)
    stretches the frequencies by ``factor`` past ``original_max_position`` as pkv_rotary_init
    describes; ``frequencies`` (radians per position, one per pair) and ``magnitude`` replace
    what that gives.  ``axes`` (one number 0..3 per pair, see :func:`rotary_axes`) says which of
    a token's positions turns each pair: rotary_and_cache then takes positions [axes, tokens]."""
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"unknown rotary scaling {scaling!r} (known: {', '.join(ROTARY_SCALINGS)})")
    r = PkvRotary()
    _check(load_library().pkv_rotary_init(ctypes.byref(r), int(rotary_dim), int(bool(interleaved)), float(base),
                                          ROTARY_SCALINGS[scaling], float(factor), int(original_max_position)))
    if frequencies is not None:
        freqs = [float(f) for f in frequencies]
        if len(freqs) != rotary_dim // 2:
            raise ValueError("frequencies must hold rotary_dim / 2 values")
        r.frequency[:len(freqs)] = freqs
    if magnitude is not None:
        r.magnitude = float(magnitude)
    if axes is not None:
        axes = [int(a) for a in axes]
        if len(axes) != rotary_dim // 2 or any(not 0 <= a <= 3 for a in axes):
            raise ValueError("axes must hold rotary_dim / 2 numbers from 0 to 3")
        r.axes = PkvRotaryAxes(max(axes, default=0) + 1)
        r.axes.axis[:len(axes)] = axes
    return r


def rotary_axes(sections, cyclic: bool = False):
    """The axis of each pair from the number of pairs that each axis has: the first
    ``sections[0]`` pairs to axis 0 and so on, or (``cyclic``) the axes in turn over the pairs
    until each has its number."""
    left = [int(n) for n in sections]
    if not 1 <= len(left) <= 4 or any(n < 0 for n in left):
        raise ValueError("sections holds one to four numbers, none below zero")
    if not cyclic:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] -= 1
    return out


def _opt_ref(t: Optional[torch.Tensor]):
    return None if t is None else _ref(t)


def rotary_and_cache(query_out, query, key, value, positions, key_cache, value_cache, slot_mapping,
                     rotary: PkvRotary, k_scale: float = 1.0, v_scale: float = 1.0, stream=None,
                     k_head_scales=None, v_head_scales=None, k_token_scales=None, v_token_scales=None) -> torch.Tensor:
    """Rotate the new tokens' queries into ``query_out`` (returned; may be ``query``) and
    write the rotated keys and the values into their cache slots, in one pass.
    ``positions`` is [tokens], or [axes, tokens] for a rotary with ``axes``.
    ``k_token_scales`` / ``v_token_scales`` go with an int8 cache ([num_blocks, Hk, block_size])
    or a 4-bit one (its group scales), which is then written as by quantize_and_cache."""
    lib = load_library()
    args = (_ref(query_out), _ref(query), _ref(key), _ref(value), _ref(positions),
            _ref(key_cache, k_scale, k_head_scales), _ref(value_cache, v_scale, v_head_scales),
            _opt_ref(k_token_scales), _opt_ref(v_token_scales), _ref(slot_mapping), ctypes.byref(rotary))
    if rotary.axes is None:
        _check(lib.pkv_rotary_and_cache(*args, _stream(stream)))
    else:
        _check(lib.pkv_rotary_axes_and_cache(*args, ctypes.byref(rotary.axes), _stream(stream)))
    return query_out


def quantize_and_cache(key, value, key_cache, value_cache, k_token_scales, v_token_scales, slot_mapping,
                       stream=None, k_scale: float = 1.0, v_scale: float = 1.0, k_head_scales=None,
                       v_head_scales=None) -> None:
    """Write the new tokens' K/V (in place) into an int8 cache, each (token, KV head) row with
    a scale of its own, max |x| / 127, stored beside the codes; or into a 4-bit cache: uint8
    [num_blocks, Hk, block_size, head_dim / 2], two e2m1 codes a byte, the scales float8_e4m3fn
    [num_blocks, Hk, block_size, head_dim / 16], one for every 16 columns.  ``k_scale`` /
    ``v_scale`` or per-head scales are a 4-bit cache's factors, the same in every call on it."""
    lib = load_library()
    _check(lib.pkv_quantize_and_cache(_ref(key), _ref(value), _ref(key_cache, k_scale, k_head_scales),
                                      _ref(value_cache, v_scale, v_head_scales), _ref(k_token_scales),
                                      _ref(v_token_scales), _ref(slot_mapping), _stream(stream)))


def read_cache(key, value, key_cache, value_cache, slot_mapping, k_scale: float = 1.0, v_scale: float = 1.0,
               stream=None, k_head_scales=None, v_head_scales=None, k_token_scales=None, v_token_scales=None):
    """Read the tokens at ``slot_mapping`` back from the cache into ``key`` and ``value``
    (float32 or bfloat16, returned); rows of negative slots stay as they were."""
    lib = load_library()
    _check(lib.pkv_read_cache(_ref(key), _ref(value), _ref(key_cache, k_scale, k_head_scales),
                              _ref(value_cache, v_scale, v_head_scales), _opt_ref(k_token_scales),
                              _opt_ref(v_token_scales), _ref(slot_mapping), _stream(stream)))
    return key, value


def paged_attention_decode_quantized(out, query, key_cache, value_cache, k_token_scales, v_token_scales, block_tables,
                                     context_lens, num_kv_heads: int, scale: float, block_size: int,
                                     max_blocks_per_seq: int, sliding_window: int = 0, stream=None,
                                     k_scale: float = 1.0, v_scale: float = 1.0, k_head_scales=None,
                                     v_head_scales=None) -> torch.Tensor:
    """Single-token decode attention over an int8 cache with one scale per (slot, KV head), or
    a 4-bit cache with its group scales (and factors, as for quantize_and_cache), into ``out``
    (returned); ``sliding_window`` as for paged_attention_decode."""
    lib = load_library()
    _check(lib.pkv_paged_attention_decode_quantized(
        _ref(out), _ref(query), _ref(key_cache, k_scale, k_head_scales), _ref(value_cache, v_scale, v_head_scales),
        _ref(k_token_scales), _ref(v_token_scales),
        _ref(block_tables), _ref(context_lens), int(num_kv_heads), float(scale), int(block_size),
        int(max_blocks_per_seq), int(sliding_window), _stream(stream)))
    return out


def paged_attention_tree(out, query, key_cache, value_cache, block_tables, context_lens, query_start_loc, tree_mask,
                         num_kv_heads: int, scale: float, block_size: int, max_blocks_per_seq: int,
                         k_scale: float = 1.0, v_scale: float = 1.0, stream=None, k_head_scales=None,
                         v_head_scales=None, k_token_scales=None, v_token_scales=None) -> torch.Tensor:
    """Attention of drafted tokens over the paged cache, into ``out`` (returned): rows
    query_start_loc[s] .. query_start_loc[s+1]-1 are sequence s's drafted nodes, the last of
    its context_lens[s] cached positions; each sees all positions before the nodes and, of
    the nodes, those whose bit is set in its row of ``tree_mask`` (int64 [rows, words])."""
    lib = load_library()
    _check(lib.pkv_paged_attention_tree(
        _ref(out), _ref(query), _ref(key_cache, k_scale, k_head_scales), _ref(value_cache, v_scale, v_head_scales),
        _opt_ref(k_token_scales), _opt_ref(v_token_scales), _ref(block_tables), _ref(context_lens),
        _ref(query_start_loc), _ref(tree_mask), int(num_kv_heads), float(scale), int(block_size),
        int(max_blocks_per_seq), _stream(stream)))
    return out


def tree_workspace_bytes(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim) -> int:
    """Most workspace bytes of a tree (or quantised decode) call with these sizes, for
    reserve_workspace before a stream capture."""
    return int(load_library().pkv_tree_workspace_bytes(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim))


def set_option(name: str, value: int) -> None:
    _check(load_library().pkv_set_option(OPTIONS[name], int(value)))


def get_option(name: str) -> int:
    return int(load_library().pkv_get_option(OPTIONS[name]))


def reserve_workspace(nbytes: int) -> None:
    _check(load_library().pkv_reserve_workspace(int(nbytes)))


def decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq) -> int:
    return int(load_library().pkv_decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                         max_blocks_per_seq))


def read_device_errors() -> int:
    """Synchronise the current device, return and clear its error word."""
    flags = ctypes.c_uint32(0)
    _check(load_library().pkv_read_device_errors(ctypes.byref(flags)))
    return int(flags.value)


def launch_count() -> int:
    return int(load_library().pkv_launch_count())


def abi_version() -> int:
    return int(load_library().pkv_abi_version())
