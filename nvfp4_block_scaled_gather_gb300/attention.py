"""ctypes binding of the attention operators of libmoe_nvfp4.so
(include/moe_attention.h): a paged cache of keys and values, the attention
that reads it, and attention over whole prompts.

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors are torch CUDA tensors; calls are enqueued on the current torch
stream (or `stream`), on the current device, whose the tensors have to be.
What torch can see of an argument (type, shape, strides, device) is checked
here and raises ValueError; a nonzero status of the library raises
RuntimeError. There is no fallback.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _native
from ._native import _check

c_int, c_size_t, c_void_p, c_longlong, c_float = (ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_longlong,
                                                  ctypes.c_float)

BF16, FP16 = 0, 1  # MOE_BF16, MOE_FP16


class Heads(ctypes.Structure):
    """moe_heads_t"""
    _fields_ = [("data", c_void_p), ("token_stride", c_longlong), ("head_stride", c_longlong)]


class CacheStruct(ctypes.Structure):
    """moe_kv_cache_t"""
    _fields_ = [("pages", c_void_p), ("planes", c_int), ("n_pages", c_int), ("page_size", c_int), ("heads_kv", c_int),
                ("head_dim", c_int), ("dtype", c_int), ("table", c_void_p), ("length", c_void_p), ("held", c_void_p),
                ("refs", c_void_p), ("max_seqs", c_int), ("max_pages", c_int)]


_CACHE, _HEADS = ctypes.POINTER(CacheStruct), c_void_p
_heads_bytes = struct.Struct("Pqq").pack  # a moe_heads_t, at a fifth of the time that the class takes

_SIGS = {
    "moe_kv_workspace_size": (c_size_t, [_CACHE]),
    "moe_kv_extend": (c_int, [_CACHE, c_void_p, c_void_p, c_int, c_void_p, c_size_t, c_void_p]),
    "moe_kv_append": (c_int, [_CACHE, c_int, c_void_p, c_void_p, c_int, c_int, _HEADS, _HEADS, c_void_p]),
    "moe_kv_fork": (c_int, [_CACHE, c_void_p, c_void_p, c_int, c_void_p]),
    "moe_kv_truncate": (c_int, [_CACHE, c_void_p, c_void_p, c_int, c_void_p]),
    "moe_kv_keep": (c_int, [_CACHE, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_int, c_void_p, c_size_t,
                            c_void_p]),
    "moe_kv_copy_pages": (c_int, [_CACHE, c_void_p, c_void_p, c_int, c_void_p]),
    "moe_kv_compact": (c_int, [_CACHE, c_void_p, c_size_t, c_void_p]),
    "moe_tree_mask": (c_int, [c_void_p, c_void_p, c_int, c_int, c_void_p, c_int, c_void_p]),
    "moe_attention_prompt": (c_int, [_HEADS, _HEADS, _HEADS, c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int,
                                     c_int, c_int, c_float, _HEADS, c_void_p, c_void_p]),
    "moe_attention_cached_workspace_size": (c_size_t, [_CACHE, c_int, c_int, c_int]),
    "moe_attention_cached": (c_int, [_HEADS, _CACHE, c_int, c_void_p, c_void_p, c_int, c_int, c_int, c_void_p, c_int,
                                     c_float, _HEADS, c_void_p, c_void_p, c_size_t, c_void_p]),
}
_LIB = None


def load():
    """The library with this header's signatures (built if stale)."""
    global _LIB
    if _LIB is None:
        lib = _native.load()
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _LIB = lib
    return _LIB


def exported_symbols():
    return list(_SIGS)


_INT32, _FLOAT32 = torch.int32, torch.float32
_MOST = 2 ** 31 - 1  # that an int of the library holds (ctypes would pass the low 32 bits on)
_CODES = {torch.bfloat16: BF16, torch.float16: FP16}


def _stream(stream, device: int) -> int:
    """The stream's handle: the given one, or the device's current one. The library launches on the current device, so
    that has to be the tensors' (the default stream's handle is the same on every device and would not tell)."""
    if torch._C._cuda_getDevice() != device:
        raise ValueError(f"tensors are on cuda:{device}, but the current device is cuda:{torch._C._cuda_getDevice()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device.index != device:
        raise ValueError(f"tensors are on cuda:{device}, but the stream's device is {stream.device}")
    return stream.cuda_stream


def _ints(name, t, n, device: int) -> int:
    """Address of a contiguous int32 tensor of n elements on this device."""
    if t.dtype is not _INT32 or t.numel() != n or not t.is_contiguous() or t.get_device() != device or device < 0:
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} elements on cuda:{device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _heads(name, t, dtype, device: int):
    """[tokens, heads, dim] with dim contiguous, as the bytes of a moe_heads_t, and its shape."""
    shape = t.shape
    if t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} on cuda:{device}, got {t.dtype} on {t.device}")
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim], got {tuple(shape)}")
    ts, hs, ds = t.stride()
    tokens, heads, dim = shape
    if tokens > _MOST or heads > _MOST:
        raise ValueError(f"{name} must have less than 2**31 tokens and heads, got {tuple(shape)}")
    # a stride along one element says nothing, and without tokens none does
    if tokens == 0:
        ts, hs, ds = 0, 0, 1
    if tokens <= 1:
        ts = 0
    if heads <= 1:
        hs = 0
    if (ds != 1 and dim != 1) or ts % 8 or hs % 8:
        raise ValueError(f"{name}: the last dimension must be contiguous and the other strides multiples of 8 elements, "
                         f"got {t.stride()}")
    return _heads_bytes(t.data_ptr(), ts, hs), shape


def _call(name, fn, *args):
    status = fn(*args)
    if status:
        _check(name, status)


class KVCache:
    """A handle over a paged cache whose memory is the caller's: pages
    [2 * layers, n_pages, page_size, kv_heads, head_dim], and int32 table
    [max_seqs, max_pages], length and held [max_seqs], refs [n_pages]
    (moe_kv_cache_t)."""

    def __init__(self, pages, table, length, held, refs):
        if pages.dim() != 5 or not pages.is_contiguous() or not pages.is_cuda or pages.dtype not in _CODES:
            raise ValueError("pages must be a contiguous bfloat16 or float16 CUDA tensor [2 * layers, n_pages, "
                             "page_size, kv_heads, head_dim]")
        if table.dim() != 2:
            raise ValueError("table must be [max_seqs, max_pages]")
        planes, n_pages, page_size, heads, dim = pages.shape
        max_seqs, max_pages = table.shape
        if max(*pages.shape, *table.shape) > _MOST:
            raise ValueError(f"pages and table must have less than 2**31 of each, got {tuple(pages.shape)} and "
                             f"{tuple(table.shape)}")
        self.pages, self.table, self.length, self.held, self.refs = pages, table, length, held, refs
        self.layers, self.device, self.dtype = planes // 2, pages.get_device(), pages.dtype
        self.heads_kv, self.head_dim, self.row = heads, dim, (heads, dim)
        self.struct = CacheStruct(pages.data_ptr(), planes, n_pages, page_size, heads, dim, _CODES[pages.dtype],
                                  _ints("table", table, max_seqs * max_pages, self.device),
                                  _ints("length", length, max_seqs, self.device),
                                  _ints("held", held, max_seqs, self.device),
                                  _ints("refs", refs, n_pages, self.device), max_seqs, max_pages)
        self._ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, layers, n_pages, page_size, kv_heads, head_dim, max_seqs, max_pages, dtype=torch.bfloat16,
              device="cuda"):
        """A fresh cache."""
        ints = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros((2 * layers, n_pages, page_size, kv_heads, head_dim), dtype=dtype, device=device),
                   torch.full((max_seqs, max_pages), -1, **ints), torch.zeros(max_seqs, **ints),
                   torch.zeros(max_seqs, **ints), torch.zeros(n_pages, **ints))


def _scratch(workspace, device: int):
    if workspace.get_device() != device or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{device}")
    return workspace.data_ptr(), workspace.numel()


def pages_workspace(cache: KVCache):
    """The scratch of moe_kv_extend, moe_kv_keep and moe_kv_compact."""
    return torch.empty(load().moe_kv_workspace_size(cache._ref), dtype=torch.uint8, device=cache.pages.device)


def moe_kv_extend(cache: KVCache, seqs, add, workspace, stream=None):
    n, dev = seqs.numel(), cache.device
    _call("moe_kv_extend", load().moe_kv_extend, cache._ref, _ints("seqs", seqs, n, dev), _ints("add", add, n, dev), n,
          *_scratch(workspace, dev), _stream(stream, dev))


def moe_kv_append(cache: KVCache, layer: int, seqs, cu, k, v, stream=None):
    n, dev = seqs.numel(), cache.device
    (hk, shape), (hv, shape_v) = _heads("k", k, cache.dtype, dev), _heads("v", v, cache.dtype, dev)
    if shape[1:] != cache.row or shape_v != shape:
        raise ValueError(f"k and v must be [total, {cache.heads_kv}, {cache.head_dim}], got {tuple(shape)} and "
                         f"{tuple(shape_v)}")
    _call("moe_kv_append", load().moe_kv_append, cache._ref, layer, _ints("seqs", seqs, n, dev),
          _ints("cu", cu, n + 1, dev), n, shape[0], hk, hv, _stream(stream, dev))


def moe_kv_fork(cache: KVCache, src, dst, stream=None):
    n, dev = src.numel(), cache.device
    _call("moe_kv_fork", load().moe_kv_fork, cache._ref, _ints("src", src, n, dev), _ints("dst", dst, n, dev), n,
          _stream(stream, dev))


def moe_kv_truncate(cache: KVCache, seqs, new_len, stream=None):
    n, dev = seqs.numel(), cache.device
    _call("moe_kv_truncate", load().moe_kv_truncate, cache._ref, _ints("seqs", seqs, n, dev),
          _ints("new_len", new_len, n, dev), n, _stream(stream, dev))


def moe_kv_keep(cache: KVCache, seqs, drafted, keep, kept, workspace, stream=None):
    n, dev = seqs.numel(), cache.device
    if keep.dim() != 2:
        raise ValueError("keep must be [n, max_keep]")
    width = keep.shape[1]
    _call("moe_kv_keep", load().moe_kv_keep, cache._ref, _ints("seqs", seqs, n, dev),
          _ints("drafted", drafted, n, dev), _ints("keep", keep, n * width, dev), width, _ints("kept", kept, n, dev), n,
          *_scratch(workspace, dev), _stream(stream, dev))


def moe_kv_copy_pages(cache: KVCache, src, dst, stream=None):
    n, dev = src.numel(), cache.device
    _call("moe_kv_copy_pages", load().moe_kv_copy_pages, cache._ref, _ints("src", src, n, dev),
          _ints("dst", dst, n, dev), n, _stream(stream, dev))


def moe_kv_compact(cache: KVCache, workspace, stream=None):
    _call("moe_kv_compact", load().moe_kv_compact, cache._ref, *_scratch(workspace, cache.device),
          _stream(stream, cache.device))


def moe_tree_mask(parents, cu, mask, stream=None):
    """mask [total, words] from the drafted tokens' parents [total]."""
    n, total, dev = cu.numel() - 1, parents.numel(), mask.get_device()
    if mask.dim() != 2:
        raise ValueError("mask must be [total, words]")
    words = mask.shape[1]
    _call("moe_tree_mask", load().moe_tree_mask, _ints("parents", parents, total, dev), _ints("cu", cu, n + 1, dev), n,
          total, _ints("mask", mask, total * words, dev), words, _stream(stream, dev))


def _lse(lse, total, heads, device: int):
    if lse is None:
        return None
    if lse.dtype is not _FLOAT32 or lse.shape != (total, heads) or not lse.is_contiguous() or lse.get_device() != device:
        raise ValueError(f"lse must be a contiguous float32 tensor {(total, heads)} on cuda:{device}")
    return lse.data_ptr()


def moe_attention_prompt(q, k, v, cu_q, cu_k, out, lse=None, scale=None, stream=None):
    """Causal attention over packed whole prompts; scale defaults to head_dim ** -0.5."""
    n, dtype, dev = cu_q.numel() - 1, q.dtype, q.get_device()
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"q must be bfloat16 or float16, got {dtype}")
    (hq, shape), (ho, shape_o) = _heads("q", q, dtype, dev), _heads("out", out, dtype, dev)
    (hk, shape_k), (hv, shape_v) = _heads("k", k, dtype, dev), _heads("v", v, dtype, dev)
    total_q, heads_q, dim = shape
    total_k, heads_kv, dim_k = shape_k
    if dim_k != dim or shape_v != shape_k or shape_o != shape:
        raise ValueError(f"k and v must be [total_k, kv_heads, {dim}] and out like q, got {tuple(shape_k)}, "
                         f"{tuple(shape_v)} and {tuple(shape_o)}")
    _call("moe_attention_prompt", load().moe_attention_prompt, hq, hk, hv,
          _ints("cu_q", cu_q, n + 1, dev), _ints("cu_k", cu_k, n + 1, dev), n, total_q, total_k, heads_q, heads_kv, dim,
          code, dim ** -0.5 if scale is None else scale, ho, _lse(lse, total_q, heads_q, dev),
          _stream(stream, dev))


def cached_workspace(cache: KVCache, n: int, total_q: int, heads_q: int):
    """The scratch of moe_attention_cached for calls of n sequences, total_q queries."""
    size = load().moe_attention_cached_workspace_size(cache._ref, n, total_q, heads_q)
    return torch.empty(size, dtype=torch.uint8, device=cache.pages.device)


def moe_attention_cached(q, cache: KVCache, layer: int, seqs, cu_q, out, workspace, mask=None, lse=None, scale=None,
                         stream=None):
    """Attention of drafted tokens (or one token a sequence) over the cache;
    mask: None for a chain, else the tree's bits (moe_tree_mask). scale
    defaults to head_dim ** -0.5."""
    n, dev = seqs.numel(), cache.device
    (hq, shape), (ho, shape_o) = _heads("q", q, cache.dtype, dev), _heads("out", out, cache.dtype, dev)
    total_q, heads_q, dim = shape
    if dim != cache.head_dim or shape_o != shape:
        raise ValueError(f"q and out must be [total_q, heads_q, {cache.head_dim}], got {tuple(shape)} and "
                         f"{tuple(shape_o)}")
    words, bits = 0, None
    if mask is not None:
        if mask.dim() != 2:
            raise ValueError("mask must be [total_q, words]")
        words = mask.shape[1]
        bits = _ints("mask", mask, total_q * words, dev)
        if words == 0 and total_q:  # (no address: the library would take it for a chain)
            raise ValueError("mask must have a word at least")
    _call("moe_attention_cached", load().moe_attention_cached, hq, cache._ref, layer,
          _ints("seqs", seqs, n, dev), _ints("cu_q", cu_q, n + 1, dev), n, total_q, heads_q, bits, words,
          dim ** -0.5 if scale is None else scale, ho, _lse(lse, total_q, heads_q, dev),
          *_scratch(workspace, dev), _stream(stream, dev))
