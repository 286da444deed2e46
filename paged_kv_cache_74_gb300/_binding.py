"""ctypes binding of libpa.so -- argument marshalling only.

Every step of the path runs in the library's CUDA kernels; these wrappers
only check tensor dtypes and shapes, turn torch tensors into device
pointers, pass torch's current CUDA stream, and raise on a non-zero
pa_status.  There is no fallback: if the library is missing, or a call is
made on tensors that are not on a CUDA device, they raise.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import builder as _build

_lock = threading.Lock()
_lib = None

PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA = range(5)
DEVICE_ERRORS = {0: "ok", 1: "bad slot", 2: "bad block id", 3: "bad seq_len",
                 4: "bad query length", 5: "wait timeout", 6: "bad rotation position",
                 7: "out of blocks", 8: "bad tree parent", 9: "bad held block count", 10: "bad accepted path"}
ABI_SYMBOLS = ("pa_status_string", "pa_abi_version", "pa_reshape_and_cache",
               "pa_compute_slot_mapping", "pa_decode_workspace_size", "pa_decode",
               "pa_prefill_workspace_size", "pa_prefill_varlen", "pa_decode_noalloc",
               "pa_map_to_kernel_blocks", "pa_reshape_and_cache_fp8", "pa_decode_fp8",
               "pa_reshape_and_cache_xsplit", "pa_decode_xsplit", "pa_append_tokens",
               "pa_reshape_and_cache_xsplit_fp8", "pa_decode_xsplit_fp8", "pa_prefill_varlen_fp8",
               "pa_qk_norm_rope_append", "pa_qk_norm_rope_append_fp8", "pa_decode_masked",
               "pa_decode_masked_fp8", "pa_prefill_masked_workspace_size", "pa_prefill_varlen_masked",
               "pa_prefill_varlen_masked_fp8", "pa_plan_step", "pa_release_blocks", "pa_commit_tokens",
               "pa_commit_planned_tokens",
               "pa_tree_workspace_size", "pa_tree_attention", "pa_tree_attention_fp8")


class PAError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed: {msg}")
        self.status = status


_i32, _i64, _sz, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float


def _declare(lib):
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_status_string.argtypes = [ctypes.c_int]
    lib.pa_abi_version.restype = ctypes.c_int
    lib.pa_abi_version.argtypes = []
    lib.pa_reshape_and_cache.restype = ctypes.c_int
    lib.pa_reshape_and_cache.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _i32, _i32,
                                         _i32, _i32, _vp, _vp]
    lib.pa_compute_slot_mapping.restype = ctypes.c_int
    lib.pa_compute_slot_mapping.argtypes = [_vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _i32,
                                            _vp, _vp]
    lib.pa_reshape_and_cache_fp8.restype = ctypes.c_int
    lib.pa_reshape_and_cache_fp8.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _i32,
                                             _i32, _i32, _i32, _f32, _f32, _vp, _vp]
    lib.pa_decode_fp8.restype = ctypes.c_int
    lib.pa_decode_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                  _i32, _i32, _i32, _f32, _f32, _f32, _i32, _vp, _sz, _vp]
    lib.pa_reshape_and_cache_xsplit.restype = ctypes.c_int
    lib.pa_reshape_and_cache_xsplit.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _i32,
                                                _i32, _i32, _i32, _vp, _vp]
    lib.pa_decode_xsplit.restype = ctypes.c_int
    lib.pa_decode_xsplit.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                     _i32, _i32, _i32, _f32, _i32, _vp, _sz, _vp]
    lib.pa_reshape_and_cache_xsplit_fp8.restype = ctypes.c_int
    lib.pa_reshape_and_cache_xsplit_fp8.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _i32,
                                                    _i32, _i32, _i32, _f32, _f32, _vp, _vp]
    lib.pa_decode_xsplit_fp8.restype = ctypes.c_int
    lib.pa_decode_xsplit_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                                         _i32, _i32, _i32, _i32, _f32, _f32, _f32, _i32, _vp, _sz,
                                         _vp]
    lib.pa_append_tokens.restype = ctypes.c_int
    lib.pa_append_tokens.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _vp, _i32,
                                     _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]
    rope = [_vp] * 4 + [_i64] * 3 + [_vp, _vp, _f32, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32,
                                     _vp, _vp] + [_i32] * 7
    lib.pa_qk_norm_rope_append.restype = ctypes.c_int
    lib.pa_qk_norm_rope_append.argtypes = rope + [_vp, _vp, _vp]
    lib.pa_qk_norm_rope_append_fp8.restype = ctypes.c_int
    lib.pa_qk_norm_rope_append_fp8.argtypes = rope + [_f32, _f32, _vp, _vp, _vp]
    lib.pa_map_to_kernel_blocks.restype = ctypes.c_int
    lib.pa_map_to_kernel_blocks.argtypes = [_vp, _vp, _i32, _i32, _i32, _vp, _vp]
    lib.pa_decode_workspace_size.restype = _sz
    lib.pa_decode_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    lib.pa_decode.restype = ctypes.c_int
    lib.pa_decode.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                              _i32, _i32, _f32, _i32, _vp, _sz, _vp]
    dec = [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32]
    lib.pa_decode_masked.restype = ctypes.c_int
    lib.pa_decode_masked.argtypes = dec + [_f32, _vp, _vp, _vp, _i32, _vp, _sz, _vp]
    lib.pa_decode_masked_fp8.restype = ctypes.c_int
    lib.pa_decode_masked_fp8.argtypes = dec + [_f32, _f32, _f32, _vp, _vp, _vp, _i32, _vp, _sz, _vp]
    lib.pa_decode_noalloc.restype = ctypes.c_int
    lib.pa_decode_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                      _i32, _i32, _i32, _f32, _i32, _vp, _vp]
    lib.pa_prefill_workspace_size.restype = _sz
    lib.pa_prefill_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    lib.pa_prefill_varlen.restype = ctypes.c_int
    lib.pa_prefill_varlen.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp,
                                      _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _sz, _vp]
    lib.pa_prefill_varlen_fp8.restype = ctypes.c_int
    lib.pa_prefill_varlen_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp,
                                          _i32, _i32, _i32, _i32, _i32, _i32, _f32, _f32, _f32, _vp,
                                          _sz, _vp]
    lib.pa_prefill_masked_workspace_size.restype = _sz
    lib.pa_prefill_masked_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    pre = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32]
    lib.pa_prefill_varlen_masked.restype = ctypes.c_int
    lib.pa_prefill_varlen_masked.argtypes = pre + [_f32, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.pa_prefill_varlen_masked_fp8.restype = ctypes.c_int
    lib.pa_prefill_varlen_masked_fp8.argtypes = pre + [_f32, _f32, _f32, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.pa_plan_step.restype = ctypes.c_int
    lib.pa_plan_step.argtypes = [_vp, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp,
                                 _i32, _vp, _vp, _i32, _vp, _vp]
    lib.pa_release_blocks.restype = ctypes.c_int
    lib.pa_release_blocks.argtypes = [_vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _vp, _vp]
    lib.pa_commit_tokens.restype = ctypes.c_int
    lib.pa_commit_tokens.argtypes = [_vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp] + [_i32] * 6 + [_vp, _vp]
    lib.pa_commit_planned_tokens.restype = ctypes.c_int
    lib.pa_commit_planned_tokens.argtypes = [_vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp] + \
        [_i32] * 6 + [_vp, _vp]
    lib.pa_tree_workspace_size.restype = _sz
    lib.pa_tree_workspace_size.argtypes = [_i32] * 6
    tree = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _vp] + [_i32] * 6 + [_f32]
    lib.pa_tree_attention.restype = ctypes.c_int
    lib.pa_tree_attention.argtypes = tree + [_vp, _sz, _vp]
    lib.pa_tree_attention_fp8.restype = ctypes.c_int
    lib.pa_tree_attention_fp8.argtypes = tree + [_f32, _f32, _vp, _sz, _vp]
    return lib


def library_path() -> str:
    return _build.LIB


def load_library(path: str | None = None):
    """Load libpa.so (built by paged_kv_cache_74_gb300.build()).  Raises if absent."""
    global _lib
    with _lock:
        if _lib is None or path is not None:
            p = path or _build.LIB
            if not os.path.exists(p):
                raise RuntimeError(f"libpa.so not built at {p}; run paged_kv_cache_74_gb300.build()")
            lib = _declare(ctypes.CDLL(p))
            if path is not None:
                return lib
            _lib = lib
        return _lib


def _check(fn, status):
    if status != PA_OK:
        raise PAError(fn, status, load_library().pa_status_string(status).decode())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _cuda(name, t, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _contig(name, t, dtype):
    _cuda(name, t, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, status=None):
    """Write key/value [T, Hkv, d] (token stride may exceed Hkv*d) into the
    caches at slot_mapping[T] (int64; negative = skip)."""
    _cuda("key", key, torch.bfloat16)
    _cuda("value", value, torch.bfloat16)
    _contig("key_cache", key_cache, torch.bfloat16)
    _contig("value_cache", value_cache, torch.bfloat16)
    _contig("slot_mapping", slot_mapping, torch.int64)
    nb, bs, hkv, d = key_cache.shape
    T = slot_mapping.shape[0]
    for name, t in (("key", key), ("value", value)):
        if tuple(t.shape) != (T, hkv, d) or t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{name} must be [T, {hkv}, {d}] with contiguous heads")
    lib = load_library()
    _check("pa_reshape_and_cache", lib.pa_reshape_and_cache(
        _ptr(key), _ptr(value), key.stride(0), value.stride(0), _ptr(key_cache),
        _ptr(value_cache), _ptr(slot_mapping), T, hkv, d, bs, nb, _ptr(status), _stream()))


def reshape_and_cache_fp8(key, value, key_cache, value_cache, slot_mapping, k_scale, v_scale,
                          status=None):
    """Quantizing write into e4m3 caches (uint8 [nb, bs, Hkv, d]): e4m3(x / scale)."""
    _cuda("key", key, torch.bfloat16)
    _cuda("value", value, torch.bfloat16)
    _contig("key_cache", key_cache, torch.uint8)
    _contig("value_cache", value_cache, torch.uint8)
    _contig("slot_mapping", slot_mapping, torch.int64)
    nb, bs, hkv, d = key_cache.shape
    T = slot_mapping.shape[0]
    for name, t in (("key", key), ("value", value)):
        if tuple(t.shape) != (T, hkv, d) or t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{name} must be [T, {hkv}, {d}] with contiguous heads")
    lib = load_library()
    _check("pa_reshape_and_cache_fp8", lib.pa_reshape_and_cache_fp8(
        _ptr(key), _ptr(value), key.stride(0), value.stride(0), _ptr(key_cache),
        _ptr(value_cache), _ptr(slot_mapping), T, hkv, d, bs, nb, float(k_scale), float(v_scale),
        _ptr(status), _stream()))


def _xsplit_shape(key_cache, value_cache):
    """(num_blocks, block_size, num_kv_heads, head_dim) of x-split caches:
    key [nb, Hkv, d / 8, bs, 8], value [nb, Hkv, d, bs]."""
    if key_cache.dim() != 5 or key_cache.shape[4] != 8:
        raise ValueError("x-split key_cache must be [num_blocks, kv_heads, head_dim / 8, block, 8]")
    nb, hkv, dx, bs, _ = key_cache.shape
    d = dx * 8
    if tuple(value_cache.shape) != (nb, hkv, d, bs):
        raise ValueError("x-split value_cache must be [num_blocks, kv_heads, head_dim, block]")
    return nb, bs, hkv, d


def reshape_and_cache_xsplit(key, value, key_cache, value_cache, slot_mapping, status=None):
    """reshape_and_cache into x-split caches (key [nb, Hkv, d / 8, bs, 8],
    value [nb, Hkv, d, bs], bf16)."""
    _cuda("key", key, torch.bfloat16)
    _cuda("value", value, torch.bfloat16)
    _contig("key_cache", key_cache, torch.bfloat16)
    _contig("value_cache", value_cache, torch.bfloat16)
    _contig("slot_mapping", slot_mapping, torch.int64)
    nb, bs, hkv, d = _xsplit_shape(key_cache, value_cache)
    T = slot_mapping.shape[0]
    for name, t in (("key", key), ("value", value)):
        if tuple(t.shape) != (T, hkv, d) or t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{name} must be [T, {hkv}, {d}] with contiguous heads")
    lib = load_library()
    _check("pa_reshape_and_cache_xsplit", lib.pa_reshape_and_cache_xsplit(
        _ptr(key), _ptr(value), key.stride(0), value.stride(0), _ptr(key_cache),
        _ptr(value_cache), _ptr(slot_mapping), T, hkv, d, bs, nb, _ptr(status), _stream()))


def _xsplit8_shape(key_cache, value_cache):
    """(num_blocks, block_size, num_kv_heads, head_dim) of e4m3 x-split caches:
    key [nb, Hkv, d / 16, bs, 16], value [nb, Hkv, d, bs] (uint8)."""
    if key_cache.dim() != 5 or key_cache.shape[4] != 16:
        raise ValueError("e4m3 x-split key_cache must be [num_blocks, kv_heads, head_dim / 16, block, 16]")
    nb, hkv, dx, bs, _ = key_cache.shape
    d = dx * 16
    if tuple(value_cache.shape) != (nb, hkv, d, bs):
        raise ValueError("e4m3 x-split value_cache must be [num_blocks, kv_heads, head_dim, block]")
    return nb, bs, hkv, d


def reshape_and_cache_xsplit_fp8(key, value, key_cache, value_cache, slot_mapping, k_scale,
                                 v_scale, status=None):
    """reshape_and_cache_fp8 into e4m3 x-split caches (key [nb, Hkv, d / 16,
    bs, 16], value [nb, Hkv, d, bs], uint8)."""
    _cuda("key", key, torch.bfloat16)
    _cuda("value", value, torch.bfloat16)
    _contig("key_cache", key_cache, torch.uint8)
    _contig("value_cache", value_cache, torch.uint8)
    _contig("slot_mapping", slot_mapping, torch.int64)
    nb, bs, hkv, d = _xsplit8_shape(key_cache, value_cache)
    T = slot_mapping.shape[0]
    for name, t in (("key", key), ("value", value)):
        if tuple(t.shape) != (T, hkv, d) or t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{name} must be [T, {hkv}, {d}] with contiguous heads")
    lib = load_library()
    _check("pa_reshape_and_cache_xsplit_fp8", lib.pa_reshape_and_cache_xsplit_fp8(
        _ptr(key), _ptr(value), key.stride(0), value.stride(0), _ptr(key_cache),
        _ptr(value_cache), _ptr(slot_mapping), T, hkv, d, bs, nb, float(k_scale), float(v_scale),
        _ptr(status), _stream()))


def compute_slot_mapping(block_tables, query_start_loc, seq_lens, block_size, num_blocks,
                         total_tokens, out=None, status=None):
    _contig("block_tables", block_tables, torch.int32)
    _contig("query_start_loc", query_start_loc, torch.int32)
    _contig("seq_lens", seq_lens, torch.int32)
    if out is None:
        out = torch.empty(total_tokens, dtype=torch.int64, device=block_tables.device)
    _contig("slot_mapping", out, torch.int64)
    lib = load_library()
    _check("pa_compute_slot_mapping", lib.pa_compute_slot_mapping(
        _ptr(out), total_tokens, _ptr(block_tables), block_tables.shape[1], _ptr(query_start_loc),
        _ptr(seq_lens), seq_lens.shape[0], block_size, num_blocks, _ptr(status), _stream()))
    return out


def append_tokens(key, value, key_cache, value_cache, block_tables, query_start_loc, seq_lens,
                  slot_mapping=None, status=None):
    """Slot mapping and cache write of the new tokens in one launch: token i of
    request r goes to the slot compute_slot_mapping gives it (slots stored in
    slot_mapping if given)."""
    _cuda("key", key, torch.bfloat16)
    _cuda("value", value, torch.bfloat16)
    _contig("key_cache", key_cache, torch.bfloat16)
    _contig("value_cache", value_cache, torch.bfloat16)
    _contig("block_tables", block_tables, torch.int32)
    _contig("query_start_loc", query_start_loc, torch.int32)
    _contig("seq_lens", seq_lens, torch.int32)
    nb, bs, hkv, d = key_cache.shape
    T = key.shape[0]
    for name, t in (("key", key), ("value", value)):
        if tuple(t.shape) != (T, hkv, d) or t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{name} must be [T, {hkv}, {d}] with contiguous heads")
    if slot_mapping is not None:
        _contig("slot_mapping", slot_mapping, torch.int64)
    lib = load_library()
    _check("pa_append_tokens", lib.pa_append_tokens(
        _ptr(key), _ptr(value), key.stride(0), value.stride(0), _ptr(key_cache), _ptr(value_cache),
        _ptr(block_tables), block_tables.shape[1], _ptr(query_start_loc), _ptr(seq_lens),
        seq_lens.shape[0], T, hkv, d, bs, nb, _ptr(slot_mapping), _ptr(status), _stream()))
    return slot_mapping


# The calls below are made for every layer of every step, often for a few
# microseconds of GPU work: their checks go over plain tuples, tensors are
# passed as integers, and the stream is read without building a Stream object.

def _fn(name):
    """The library's function of that name (loaded on first use)."""
    return getattr(_lib if _lib is not None else load_library(), name)


def _refuse(name, t, dtype, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _check_all(dev, needed, optional):
    """Every (name, tensor, dtype) a contiguous CUDA tensor of device `dev`, the
    optional ones or None."""
    for name, t, dtype in needed:
        if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or \
                not t.is_contiguous():
            _refuse(name, t, dtype, dev)
    for name, t, dtype in optional:
        if t is not None and (not isinstance(t, torch.Tensor) or t.dtype is not dtype or
                              t.get_device() != dev or not t.is_contiguous()):
            _refuse(name, t, dtype, dev)


def _device_of(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _addr(t):
    return t.data_ptr() if t is not None else 0


def _launch(name, dev, *args):
    """Calls the library with `dev` current, on its current stream."""
    fn = _fn(name)
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status != PA_OK:
        _check(name, status)


def _heads(name, t, dev, T, heads, d):
    """The token stride of t [T, heads, d].  One token has none of its own (torch
    leaves that stride arbitrary): a row's size then."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.get_device() != dev:
        _refuse(name, t, torch.bfloat16, dev)
    stride = t.stride()
    if t.shape != (T, heads, d) or stride[2] != 1 or (stride[1] != d and heads > 1):
        raise ValueError(f"{name} must be [{T}, {heads}, {d}] with contiguous heads")
    return stride[0] if T != 1 else heads * d


def _qk_norm_rope(fn, cache_dtype, scales, q, key, value, key_cache, value_cache, block_tables,
                  query_start_loc, seq_lens, cos_sin, q_weight, k_weight, eps, interleaved, positions,
                  out, slot_mapping, status):
    dev = _device_of("q", q)
    i32 = torch.int32
    _check_all(dev, (("key_cache", key_cache, cache_dtype), ("value_cache", value_cache, cache_dtype),
                     ("block_tables", block_tables, i32), ("query_start_loc", query_start_loc, i32),
                     ("seq_lens", seq_lens, i32), ("cos_sin", cos_sin, torch.float32)),
               (("q_weight", q_weight, torch.float32), ("k_weight", k_weight, torch.float32),
                ("positions", positions, i32), ("out", out, torch.bfloat16),
                ("slot_mapping", slot_mapping, torch.int64), ("status", status, i32)))
    if key_cache.dim() != 4 or value_cache.shape != key_cache.shape:
        raise ValueError("key_cache and value_cache must be [num_blocks, block, kv_heads, head_dim]")
    nb, bs, hkv, d = key_cache.shape
    if q.dim() != 3:
        raise ValueError("q must be [T, heads, head_dim]")
    T, hq, _ = q.shape
    qs = _heads("q", q, dev, T, hq, d)
    ks = _heads("key", key, dev, T, hkv, d)
    vs = _heads("value", value, dev, T, hkv, d)
    S = seq_lens.shape[0]
    if block_tables.dim() != 2 or block_tables.shape[0] != S or query_start_loc.shape[0] != S + 1:
        raise ValueError("block_tables must be [num_seqs, max_blocks] and query_start_loc [num_seqs + 1]")
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_position, rot_dim]")
    for name, t, n in (("q_weight", q_weight, d), ("k_weight", k_weight, d), ("positions", positions, T),
                       ("slot_mapping", slot_mapping, T)):
        if t is not None and t.numel() != n:
            raise ValueError(f"{name} must be [{n}]")
    if status is not None and status.numel() < 4:
        raise ValueError("status must hold 4 values")
    if out is None:
        out = torch.empty((T, hq, d), dtype=torch.bfloat16, device=q.device)
    elif out.shape != q.shape:
        raise ValueError(f"out must be [{T}, {hq}, {d}]")
    _launch(fn, dev, out.data_ptr(), q.data_ptr(), key.data_ptr(), value.data_ptr(), qs, ks, vs,
            _addr(q_weight), _addr(k_weight), float(eps), cos_sin.data_ptr(), cos_sin.shape[0],
            cos_sin.shape[1], 1 if interleaved else 0, _addr(positions), key_cache.data_ptr(),
            value_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
            query_start_loc.data_ptr(), seq_lens.data_ptr(), S, T, hq, hkv, d, bs, nb, *scales,
            _addr(slot_mapping), _addr(status))
    return out


def qk_norm_rope_append(q, key, value, key_cache, value_cache, block_tables, query_start_loc, seq_lens,
                        cos_sin, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                        positions=None, out=None, slot_mapping=None, status=None):
    """Norm of every q and k head (float weights [d]; None: not normed), rotation
    by the rows of cos_sin [max_position, rot_dim] (rot_dim / 2 cosines, then
    sines), and the cache write of append_tokens, in one launch.  Returns the
    normed, rotated q [T, Hq, d] (out may be q itself if q is contiguous).
    positions: rotation positions [T] int32 (None: the tokens' positions in
    their requests)."""
    return _qk_norm_rope("pa_qk_norm_rope_append", torch.bfloat16, (), q, key, value, key_cache,
                         value_cache, block_tables, query_start_loc, seq_lens, cos_sin, q_weight,
                         k_weight, eps, interleaved, positions, out, slot_mapping, status)


def qk_norm_rope_append_fp8(q, key, value, key_cache, value_cache, block_tables, query_start_loc,
                            seq_lens, cos_sin, k_scale, v_scale, q_weight=None, k_weight=None, eps=1e-6,
                            interleaved=False, positions=None, out=None, slot_mapping=None, status=None):
    """qk_norm_rope_append into e4m3 caches (uint8 [nb, bs, Hkv, d]): e4m3(x / scale)."""
    return _qk_norm_rope("pa_qk_norm_rope_append_fp8", torch.uint8, (float(k_scale), float(v_scale)), q,
                         key, value, key_cache, value_cache, block_tables, query_start_loc, seq_lens,
                         cos_sin, q_weight, k_weight, eps, interleaved, positions, out, slot_mapping,
                         status)


def map_to_kernel_blocks(block_tables, blocks_per_kv_block, out=None, status=None):
    """Block tables of manager blocks -> tables of kernel blocks (k per manager block)."""
    _contig("block_tables", block_tables, torch.int32)
    rows, cols = block_tables.shape
    k = int(blocks_per_kv_block)
    if out is None:
        out = torch.empty((rows, cols * k), dtype=torch.int32, device=block_tables.device)
    _contig("kernel_tables", out, torch.int32)
    lib = load_library()
    _check("pa_map_to_kernel_blocks", lib.pa_map_to_kernel_blocks(
        _ptr(out), _ptr(block_tables), rows, cols, k, _ptr(status), _stream()))
    return out


def decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len,
                          partition_tokens=0):
    return int(load_library().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                       max_seq_len, partition_tokens))


def new_workspace(nbytes, device):
    """A zeroed workspace (the status record starts clean)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def decode(q, key_cache, value_cache, block_tables, seq_lens, max_seq_len, scale, out=None,
           workspace=None, partition_tokens=0):
    """Paged decode attention; q [S, Hq, d] -> out [S, Hq, d] (bf16)."""
    _contig("q", q, torch.bfloat16)
    _contig("key_cache", key_cache, torch.bfloat16)
    _contig("value_cache", value_cache, torch.bfloat16)
    _contig("block_tables", block_tables, torch.int32)
    _contig("seq_lens", seq_lens, torch.int32)
    S, hq, d = q.shape
    nb, bs, hkv, d2 = key_cache.shape
    if d2 != d or value_cache.shape != key_cache.shape:
        raise ValueError("cache shapes do not match q")
    if out is None:
        out = torch.empty_like(q)
    _contig("out", out, torch.bfloat16)
    if workspace is None:
        workspace = new_workspace(decode_workspace_size(S, hq, hkv, d, max_seq_len, partition_tokens),
                                  q.device)
    lib = load_library()
    _check("pa_decode", lib.pa_decode(
        _ptr(out), _ptr(q), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), S, int(max_seq_len), hq, hkv, d, bs, nb,
        float(scale), int(partition_tokens), _ptr(workspace), workspace.numel(), _stream()))
    return out


def decode_fp8(q, key_cache, value_cache, block_tables, seq_lens, max_seq_len, scale, k_scale,
               v_scale, out=None, workspace=None, partition_tokens=0):
    """Paged decode over e4m3 caches (uint8 [nb, bs, Hkv, d]); q, out bf16."""
    _contig("q", q, torch.bfloat16)
    _contig("key_cache", key_cache, torch.uint8)
    _contig("value_cache", value_cache, torch.uint8)
    _contig("block_tables", block_tables, torch.int32)
    _contig("seq_lens", seq_lens, torch.int32)
    S, hq, d = q.shape
    nb, bs, hkv, d2 = key_cache.shape
    if d2 != d or value_cache.shape != key_cache.shape:
        raise ValueError("cache shapes do not match q")
    if out is None:
        out = torch.empty_like(q)
    _contig("out", out, torch.bfloat16)
    if workspace is None:
        workspace = new_workspace(decode_workspace_size(S, hq, hkv, d, max_seq_len, partition_tokens),
                                  q.device)
    lib = load_library()
    _check("pa_decode_fp8", lib.pa_decode_fp8(
        _ptr(out), _ptr(q), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), S, int(max_seq_len), hq, hkv, d, bs, nb,
        float(scale), float(k_scale), float(v_scale), int(partition_tokens), _ptr(workspace),
        workspace.numel(), _stream()))
    return out


def decode_xsplit(q, key_cache, value_cache, block_tables, seq_lens, max_seq_len, scale,
                  out=None, workspace=None, partition_tokens=0):
    """Paged decode over x-split caches (see reshape_and_cache_xsplit)."""
    _contig("q", q, torch.bfloat16)
    _contig("key_cache", key_cache, torch.bfloat16)
    _contig("value_cache", value_cache, torch.bfloat16)
    _contig("block_tables", block_tables, torch.int32)
    _contig("seq_lens", seq_lens, torch.int32)
    S, hq, d = q.shape
    nb, bs, hkv, d2 = _xsplit_shape(key_cache, value_cache)
    if d2 != d:
        raise ValueError("cache shapes do not match q")
    if out is None:
        out = torch.empty_like(q)
    _contig("out", out, torch.bfloat16)
    if workspace is None:
        workspace = new_workspace(decode_workspace_size(S, hq, hkv, d, max_seq_len, partition_tokens),
                                  q.device)
    lib = load_library()
    _check("pa_decode_xsplit", lib.pa_decode_xsplit(
        _ptr(out), _ptr(q), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), S, int(max_seq_len), hq, hkv, d, bs, nb,
        float(scale), int(partition_tokens), _ptr(workspace), workspace.numel(), _stream()))
    return out


def decode_xsplit_fp8(q, key_cache, value_cache, block_tables, seq_lens, max_seq_len, scale,
                      k_scale, v_scale, out=None, workspace=None, partition_tokens=0):
    """Paged decode over e4m3 x-split caches (see reshape_and_cache_xsplit_fp8)."""
    _contig("q", q, torch.bfloat16)
    _contig("key_cache", key_cache, torch.uint8)
    _contig("value_cache", value_cache, torch.uint8)
    _contig("block_tables", block_tables, torch.int32)
    _contig("seq_lens", seq_lens, torch.int32)
    S, hq, d = q.shape
    nb, bs, hkv, d2 = _xsplit8_shape(key_cache, value_cache)
    if d2 != d:
        raise ValueError("cache shapes do not match q")
    if out is None:
        out = torch.empty_like(q)
    _contig("out", out, torch.bfloat16)
    if workspace is None:
        workspace = new_workspace(decode_workspace_size(S, hq, hkv, d, max_seq_len, partition_tokens),
                                  q.device)
    lib = load_library()
    _check("pa_decode_xsplit_fp8", lib.pa_decode_xsplit_fp8(
        _ptr(out), _ptr(q), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), S, int(max_seq_len), hq, hkv, d, bs, nb,
        float(scale), float(k_scale), float(v_scale), int(partition_tokens), _ptr(workspace),
        workspace.numel(), _stream()))
    return out


def decode_noalloc(q, key_cache, value_cache, block_tables, seq_lens, max_seq_len, scale,
                   out=None, partition_tokens=0, status=None):
    """pa_decode without a workspace: for callers that cannot allocate device
    memory.  Scratch comes from a fixed-size array inside the library (see
    include/pa.h); calls that overlap on the GPU must be serialised.  status:
    optional int32[4] CUDA tensor that receives the call's device status
    record."""
    _contig("q", q, torch.bfloat16)
    _contig("key_cache", key_cache, torch.bfloat16)
    _contig("value_cache", value_cache, torch.bfloat16)
    _contig("block_tables", block_tables, torch.int32)
    _contig("seq_lens", seq_lens, torch.int32)
    S, hq, d = q.shape
    nb, bs, hkv, _ = key_cache.shape
    if out is None:
        out = torch.empty_like(q)
    _contig("out", out, torch.bfloat16)
    lib = load_library()
    _check("pa_decode_noalloc", lib.pa_decode_noalloc(
        _ptr(out), _ptr(q), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), S, int(max_seq_len), hq, hkv, d, bs, nb,
        float(scale), int(partition_tokens), _ptr(status), _stream()))
    return out


def _attention_args(q, key_cache, value_cache, cache_dtype, block_tables, seq_lens, out, slopes,
                    key_starts, prefix_lens, workspace, query_start_loc):
    """Checks shared by the masked attention calls; returns (device index, out)."""
    dev = _device_of("q", q)
    bf16, i32 = torch.bfloat16, torch.int32
    _check_all(dev, (("q", q, bf16), ("key_cache", key_cache, cache_dtype),
                     ("value_cache", value_cache, cache_dtype), ("block_tables", block_tables, i32),
                     ("seq_lens", seq_lens, i32)),
               (("query_start_loc", query_start_loc, i32), ("out", out, bf16),
                ("slopes", slopes, torch.float32), ("key_starts", key_starts, i32),
                ("prefix_lens", prefix_lens, i32), ("workspace", workspace, torch.uint8)))
    if q.dim() != 3 or key_cache.dim() != 4 or key_cache.shape[3] != q.shape[2] or \
            value_cache.shape != key_cache.shape:
        raise ValueError("cache shapes do not match q")
    S = seq_lens.shape[0]
    if block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("block_tables must be [num_seqs, max_blocks]")
    rows, hq = q.shape[0], q.shape[1]
    if slopes is not None and slopes.numel() != hq:
        raise ValueError(f"slopes must be [{hq}]")
    if key_starts is not None and key_starts.numel() != rows:
        raise ValueError(f"key_starts must be [{rows}]")
    if prefix_lens is not None and prefix_lens.numel() != S:
        raise ValueError(f"prefix_lens must be [{S}]")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    return dev, out


def _decode_masked(fn, cache_dtype, scales, q, key_cache, value_cache, block_tables, seq_lens,
                   max_seq_len, scale, softcap, slopes, key_starts, prefix_lens, out, workspace,
                   partition_tokens):
    dev, out = _attention_args(q, key_cache, value_cache, cache_dtype, block_tables, seq_lens, out,
                               slopes, key_starts, prefix_lens, workspace, None)
    S, hq, d = q.shape
    nb, bs, hkv, _ = key_cache.shape
    if seq_lens.shape[0] != S:
        raise ValueError(f"seq_lens must be [{S}]")
    if workspace is None:
        with torch.cuda.device(dev):
            workspace = new_workspace(
                decode_workspace_size(S, hq, hkv, d, max_seq_len, partition_tokens), q.device)
    _launch(fn, dev, out.data_ptr(), q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
            block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(), S, int(max_seq_len), hq,
            hkv, d, bs, nb, float(scale), *scales, float(softcap), _addr(slopes), _addr(key_starts),
            _addr(prefix_lens), int(partition_tokens), workspace.data_ptr(), workspace.numel())
    return out


def decode_masked(q, key_cache, value_cache, block_tables, seq_lens, max_seq_len, scale, softcap=0.0,
                  slopes=None, key_starts=None, prefix_lens=None, out=None, workspace=None,
                  partition_tokens=0):
    """Paged decode with modified scores: s = scale q.k, then softcap tanh(s /
    softcap) (0: none), then - slopes[h] |p - j| (float [Hq]); a row sees keys
    j < prefix_lens[r] (int32 [S]) and key_starts[row] <= j <= p (int32 [S]).
    A row that sees no key gives zeros."""
    return _decode_masked("pa_decode_masked", torch.bfloat16, (), q, key_cache, value_cache, block_tables,
                          seq_lens, max_seq_len, scale, softcap, slopes, key_starts, prefix_lens, out,
                          workspace, partition_tokens)


def decode_masked_fp8(q, key_cache, value_cache, block_tables, seq_lens, max_seq_len, scale, k_scale,
                      v_scale, softcap=0.0, slopes=None, key_starts=None, prefix_lens=None, out=None,
                      workspace=None, partition_tokens=0):
    """decode_masked over e4m3 caches (uint8 [nb, bs, Hkv, d]) with their scales."""
    return _decode_masked("pa_decode_masked_fp8", torch.uint8, (float(k_scale), float(v_scale)), q,
                          key_cache, value_cache, block_tables, seq_lens, max_seq_len, scale, softcap,
                          slopes, key_starts, prefix_lens, out, workspace, partition_tokens)


def prefill_workspace_size(num_seqs, total_q, num_heads, num_kv_heads, head_dim, max_seq_len):
    return int(load_library().pa_prefill_workspace_size(num_seqs, total_q, num_heads, num_kv_heads,
                                                        head_dim, max_seq_len))


def prefill_varlen(q, key_cache, value_cache, query_start_loc, seq_lens, block_tables,
                   max_query_len, max_seq_len, scale, out=None, workspace=None):
    """Mixed chunked-prefill + decode attention; q [total_q, Hq, d]."""
    _contig("q", q, torch.bfloat16)
    _contig("key_cache", key_cache, torch.bfloat16)
    _contig("value_cache", value_cache, torch.bfloat16)
    _contig("query_start_loc", query_start_loc, torch.int32)
    _contig("seq_lens", seq_lens, torch.int32)
    _contig("block_tables", block_tables, torch.int32)
    tq, hq, d = q.shape
    nb, bs, hkv, _ = key_cache.shape
    S = seq_lens.shape[0]
    if out is None:
        out = torch.empty_like(q)
    _contig("out", out, torch.bfloat16)
    if workspace is None:
        workspace = new_workspace(prefill_workspace_size(S, tq, hq, hkv, d, max_seq_len), q.device)
    lib = load_library()
    _check("pa_prefill_varlen", lib.pa_prefill_varlen(
        _ptr(out), _ptr(q), _ptr(key_cache), _ptr(value_cache), _ptr(query_start_loc),
        _ptr(seq_lens), S, tq, int(max_query_len), int(max_seq_len), _ptr(block_tables),
        block_tables.shape[1], hq, hkv, d, bs, nb, float(scale), _ptr(workspace),
        workspace.numel(), _stream()))
    return out


def prefill_varlen_fp8(q, key_cache, value_cache, query_start_loc, seq_lens, block_tables,
                       max_query_len, max_seq_len, scale, k_scale, v_scale, out=None, workspace=None):
    """prefill_varlen over e4m3 caches (uint8 [nb, bs, Hkv, d]) with their scales."""
    _contig("q", q, torch.bfloat16)
    _contig("key_cache", key_cache, torch.uint8)
    _contig("value_cache", value_cache, torch.uint8)
    _contig("query_start_loc", query_start_loc, torch.int32)
    _contig("seq_lens", seq_lens, torch.int32)
    _contig("block_tables", block_tables, torch.int32)
    tq, hq, d = q.shape
    nb, bs, hkv, d2 = key_cache.shape
    if d2 != d or value_cache.shape != key_cache.shape:
        raise ValueError("cache shapes do not match q")
    S = seq_lens.shape[0]
    if out is None:
        out = torch.empty_like(q)
    _contig("out", out, torch.bfloat16)
    if workspace is None:
        workspace = new_workspace(prefill_workspace_size(S, tq, hq, hkv, d, max_seq_len), q.device)
    lib = load_library()
    _check("pa_prefill_varlen_fp8", lib.pa_prefill_varlen_fp8(
        _ptr(out), _ptr(q), _ptr(key_cache), _ptr(value_cache), _ptr(query_start_loc),
        _ptr(seq_lens), S, tq, int(max_query_len), int(max_seq_len), _ptr(block_tables),
        block_tables.shape[1], hq, hkv, d, bs, nb, float(scale), float(k_scale), float(v_scale),
        _ptr(workspace), workspace.numel(), _stream()))
    return out


def prefill_masked_workspace_size(num_seqs, total_q, num_heads, num_kv_heads, head_dim, max_seq_len):
    return int(load_library().pa_prefill_masked_workspace_size(num_seqs, total_q, num_heads,
                                                               num_kv_heads, head_dim, max_seq_len))


def _prefill_masked(fn, cache_dtype, scales, q, key_cache, value_cache, query_start_loc, seq_lens,
                    block_tables, max_query_len, max_seq_len, scale, softcap, slopes, key_starts,
                    prefix_lens, out, workspace):
    dev, out = _attention_args(q, key_cache, value_cache, cache_dtype, block_tables, seq_lens, out,
                               slopes, key_starts, prefix_lens, workspace, query_start_loc)
    tq, hq, d = q.shape
    nb, bs, hkv, _ = key_cache.shape
    S = seq_lens.shape[0]
    if query_start_loc is None or query_start_loc.numel() != S + 1:
        raise ValueError(f"query_start_loc must be [{S + 1}]")
    if workspace is None:
        with torch.cuda.device(dev):
            workspace = new_workspace(prefill_masked_workspace_size(S, tq, hq, hkv, d, max_seq_len),
                                      q.device)
    _launch(fn, dev, out.data_ptr(), q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
            query_start_loc.data_ptr(), seq_lens.data_ptr(), S, tq, int(max_query_len), int(max_seq_len),
            block_tables.data_ptr(), block_tables.shape[1], hq, hkv, d, bs, nb, float(scale), *scales,
            float(softcap), _addr(slopes), _addr(key_starts), _addr(prefix_lens), workspace.data_ptr(),
            workspace.numel())
    return out


def prefill_varlen_masked(q, key_cache, value_cache, query_start_loc, seq_lens, block_tables,
                          max_query_len, max_seq_len, scale, softcap=0.0, slopes=None, key_starts=None,
                          prefix_lens=None, out=None, workspace=None):
    """prefill_varlen with the modified scores of decode_masked: softcap, slopes
    [Hq], key_starts [total_q] (one per query row) and prefix_lens [S], whose
    keys every row of the request sees, also the rows before them."""
    return _prefill_masked("pa_prefill_varlen_masked", torch.bfloat16, (), q, key_cache, value_cache,
                           query_start_loc, seq_lens, block_tables, max_query_len, max_seq_len, scale,
                           softcap, slopes, key_starts, prefix_lens, out, workspace)


def prefill_varlen_masked_fp8(q, key_cache, value_cache, query_start_loc, seq_lens, block_tables,
                              max_query_len, max_seq_len, scale, k_scale, v_scale, softcap=0.0,
                              slopes=None, key_starts=None, prefix_lens=None, out=None, workspace=None):
    """prefill_varlen_masked over e4m3 caches (uint8 [nb, bs, Hkv, d]) with their scales."""
    return _prefill_masked("pa_prefill_varlen_masked_fp8", torch.uint8, (float(k_scale), float(v_scale)), q,
                           key_cache, value_cache, query_start_loc, seq_lens, block_tables,
                           max_query_len, max_seq_len, scale, softcap, slopes, key_starts, prefix_lens,
                           out, workspace)


def tree_workspace_size(num_seqs, total_q, num_heads, num_kv_heads, head_dim, max_seq_len):
    return int(load_library().pa_tree_workspace_size(num_seqs, total_q, num_heads, num_kv_heads, head_dim,
                                                     max_seq_len))


def _tree_attention(fn, cache_dtype, scales, q, key_cache, value_cache, query_start_loc, seq_lens,
                    block_tables, tree_masks, max_query_len, max_seq_len, scale, out, workspace):
    dev = _device_of("q", q)
    bf16, i32 = torch.bfloat16, torch.int32
    _check_all(dev, (("q", q, bf16), ("key_cache", key_cache, cache_dtype),
                     ("value_cache", value_cache, cache_dtype), ("query_start_loc", query_start_loc, i32),
                     ("seq_lens", seq_lens, i32), ("block_tables", block_tables, i32),
                     ("tree_masks", tree_masks, torch.int64)),
               (("out", out, bf16), ("workspace", workspace, torch.uint8)))
    q_shape, shape = q.shape, key_cache.shape
    if len(q_shape) != 3 or len(shape) != 4 or shape[3] != q_shape[2] or value_cache.shape != shape:
        raise ValueError("cache shapes do not match q")
    tq, hq, d = q_shape
    nb, bs, hkv, _ = shape
    S, width = _table_shape(block_tables)
    if seq_lens.numel() != S or query_start_loc.numel() != S + 1:
        raise ValueError(f"seq_lens must be [{S}] and query_start_loc [{S + 1}]")
    words = _mask_words(tree_masks, tq)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q_shape:
        raise ValueError("out must have q's shape")
    if tq == 0 or S == 0:
        return out
    if workspace is None:
        with torch.cuda.device(dev):
            workspace = new_workspace(tree_workspace_size(S, tq, hq, hkv, d, max_seq_len), q.device)
    _launch(fn, dev, out.data_ptr(), q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
            query_start_loc.data_ptr(), seq_lens.data_ptr(), S, tq, int(max_query_len), int(max_seq_len),
            block_tables.data_ptr(), width, tree_masks.data_ptr(), words, hq, hkv, d, bs, nb,
            float(scale), *scales, workspace.data_ptr(), workspace.numel())
    return out


def tree_attention(q, key_cache, value_cache, query_start_loc, seq_lens, block_tables, tree_masks,
                   max_query_len, max_seq_len, scale, out=None, workspace=None):
    """Attention of drafted token trees; q [total_q, Hq, d] packed by query_start_loc.
    A row sees its request's context (the seq_len - q_len keys before the rows') and
    the rows named by its bits of tree_masks (int64 [total_q, words] or [total_q], as
    plan_step writes them).  A row that sees no key gives zeros."""
    return _tree_attention("pa_tree_attention", torch.bfloat16, (), q, key_cache, value_cache,
                           query_start_loc, seq_lens, block_tables, tree_masks, max_query_len, max_seq_len,
                           scale, out, workspace)


def tree_attention_fp8(q, key_cache, value_cache, query_start_loc, seq_lens, block_tables, tree_masks,
                       max_query_len, max_seq_len, scale, k_scale, v_scale, out=None, workspace=None):
    """tree_attention over e4m3 caches (uint8 [nb, bs, Hkv, d]) with their scales."""
    return _tree_attention("pa_tree_attention_fp8", torch.uint8, (float(k_scale), float(v_scale)), q, key_cache,
                           value_cache, query_start_loc, seq_lens, block_tables, tree_masks, max_query_len,
                           max_seq_len, scale, out, workspace)


def _lens(S, *named):
    for name, t in named:
        if t.numel() != S:
            raise ValueError(f"{name} must be [{S}]")


def _status4(status):
    if status.numel() < 4:
        raise ValueError("status must hold 4 values")


def _table_shape(block_tables):
    shape = block_tables.shape
    if len(shape) != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks]")
    return shape


def _mask_words(tree_masks, rows):
    shape = tree_masks.shape
    if len(shape) not in (1, 2) or shape[0] != rows:
        raise ValueError(f"tree_masks must be [{rows}, words]")
    return shape[1] if len(shape) == 2 else 1


def plan_step(block_tables, held_blocks, context_lens, query_lens, free_blocks, free_count, block_size,
              num_blocks, query_start_loc, seq_lens, slot_mapping, positions, parents=None, tree_masks=None,
              status=None):
    """The step's bookkeeping on the device, from the requests' lengths (int32 [S]):
    new blocks off the end of free_blocks [capacity] (free_count [1] of them valid)
    into block_tables [S, max_blocks] behind held_blocks [S]; query_start_loc
    [S + 1], seq_lens [S], slot_mapping (int64) and positions (int32) [max_tokens];
    with tree_masks (int64 [max_tokens, words] or [max_tokens]) the ancestors' bits of
    each row, from parents [max_tokens] (-1: follows the context; None: a chain).
    Returns (query_start_loc, seq_lens, slot_mapping, positions, tree_masks)."""
    dev = _device_of("block_tables", block_tables)
    i32, i64 = torch.int32, torch.int64
    _check_all(dev, (("block_tables", block_tables, i32), ("held_blocks", held_blocks, i32),
                     ("context_lens", context_lens, i32), ("query_lens", query_lens, i32),
                     ("free_blocks", free_blocks, i32), ("free_count", free_count, i32),
                     ("query_start_loc", query_start_loc, i32), ("seq_lens", seq_lens, i32),
                     ("slot_mapping", slot_mapping, i64), ("positions", positions, i32)),
               (("parents", parents, i32), ("tree_masks", tree_masks, i64), ("status", status, i32)))
    S, width = _table_shape(block_tables)
    T = slot_mapping.numel()
    if not held_blocks.numel() == context_lens.numel() == query_lens.numel() == seq_lens.numel() == S:
        _lens(S, ("held_blocks", held_blocks), ("context_lens", context_lens), ("query_lens", query_lens),
              ("seq_lens", seq_lens))
    if positions.numel() != T:
        raise ValueError(f"positions must be [{T}]")
    if query_start_loc.numel() != S + 1 or free_count.numel() != 1:
        raise ValueError(f"query_start_loc must be [{S + 1}] and free_count [1]")
    if parents is not None and parents.numel() != T:
        raise ValueError(f"parents must be [{T}]")
    words = _mask_words(tree_masks, T) if tree_masks is not None else 0
    if status is not None:
        _status4(status)
    _launch("pa_plan_step", dev, block_tables.data_ptr(), width, held_blocks.data_ptr(),
            context_lens.data_ptr(), query_lens.data_ptr(), S, free_blocks.data_ptr(), free_blocks.numel(),
            free_count.data_ptr(), int(block_size), int(num_blocks), query_start_loc.data_ptr(),
            seq_lens.data_ptr(), slot_mapping.data_ptr(), positions.data_ptr(), T, _addr(parents),
            _addr(tree_masks), words, _addr(status))
    return query_start_loc, seq_lens, slot_mapping, positions, tree_masks


def release_blocks(block_tables, held_blocks, keep_lens, free_blocks, free_count, block_size, num_blocks,
                   status=None):
    """Gives the blocks of each request behind its first keep_lens [S] tokens (0: all)
    back to the list of plan_step; held_blocks becomes what is left."""
    dev = _device_of("block_tables", block_tables)
    i32 = torch.int32
    _check_all(dev, (("block_tables", block_tables, i32), ("held_blocks", held_blocks, i32),
                     ("keep_lens", keep_lens, i32), ("free_blocks", free_blocks, i32),
                     ("free_count", free_count, i32)), (("status", status, i32),))
    S, width = _table_shape(block_tables)
    if not held_blocks.numel() == keep_lens.numel() == S:
        _lens(S, ("held_blocks", held_blocks), ("keep_lens", keep_lens))
    if free_count.numel() != 1:
        raise ValueError("free_count must be [1]")
    if status is not None:
        _status4(status)
    _launch("pa_release_blocks", dev, block_tables.data_ptr(), width, held_blocks.data_ptr(),
            keep_lens.data_ptr(), S, free_blocks.data_ptr(), free_blocks.numel(), free_count.data_ptr(),
            int(block_size), int(num_blocks), _addr(status))


def commit_tokens(key_cache, value_cache, block_tables, context_lens, query_lens, accepted, accept_lens,
                  new_lens=None, status=None, seq_lens=None):
    """Moves K and V of the accepted rows (accepted int32 [S, max_accepted], ascending,
    the first accept_lens [S] of them) to the slots behind context_lens [S], in caches
    [num_blocks, block, kv_heads, head_dim] or [layers, num_blocks, ..] (bf16 or
    uint8).  Returns new_lens [S] = context_lens + accept_lens.  With seq_lens [S], as
    plan_step wrote them, requests that the plan refused are left alone (new_lens =
    context_lens); without, their accept_lens must be 0."""
    dev = _device_of("key_cache", key_cache)
    i32 = torch.int32
    dtype = torch.uint8 if key_cache.dtype is torch.uint8 else torch.bfloat16
    _check_all(dev, (("key_cache", key_cache, dtype), ("value_cache", value_cache, dtype),
                     ("block_tables", block_tables, i32), ("context_lens", context_lens, i32),
                     ("query_lens", query_lens, i32), ("accepted", accepted, i32),
                     ("accept_lens", accept_lens, i32)), (("new_lens", new_lens, i32), ("status", status, i32),
                                                        ("seq_lens", seq_lens, i32)))
    shape = key_cache.shape
    if len(shape) not in (4, 5) or value_cache.shape != shape:
        raise ValueError("key_cache and value_cache must be [(layers,) num_blocks, block, kv_heads, head_dim]")
    layers, nb, bs, hkv, d = shape if len(shape) == 5 else (1, *shape)
    if layers == 0:
        raise ValueError("key_cache and value_cache must hold a layer")
    S, width = _table_shape(block_tables)
    path = accepted.shape
    if len(path) != 2 or path[0] != S:
        raise ValueError(f"accepted must be [{S}, max_accepted]")
    if new_lens is None:
        new_lens = torch.empty_like(context_lens)
    if not context_lens.numel() == query_lens.numel() == accept_lens.numel() == new_lens.numel() == S:
        _lens(S, ("context_lens", context_lens), ("query_lens", query_lens), ("accept_lens", accept_lens),
              ("new_lens", new_lens))
    if status is not None:
        _status4(status)
    fn, planned = "pa_commit_tokens", ()
    if seq_lens is not None:
        _lens(S, ("seq_lens", seq_lens))
        fn, planned = "pa_commit_planned_tokens", (seq_lens.data_ptr(),)
    _launch(fn, dev, key_cache.data_ptr(), value_cache.data_ptr(), layers, block_tables.data_ptr(),
            width, context_lens.data_ptr(), query_lens.data_ptr(), *planned, accepted.data_ptr(),
            path[1], accept_lens.data_ptr(), new_lens.data_ptr(), S, hkv, d, bs, nb,
            1 if dtype is torch.uint8 else 2, _addr(status))
    return new_lens


def device_status(workspace_or_status):
    """Read the int32[4] device status record (synchronises the stream)."""
    t = workspace_or_status
    rec = t[:16].view(torch.int32) if t.dtype == torch.uint8 else t[:4]
    return [int(x) for x in rec.cpu()]
