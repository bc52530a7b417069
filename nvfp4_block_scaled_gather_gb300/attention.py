"""ctypes binding of the attention operators of libmoe_nvfp4.so
(include/moe_attention.h): a paged cache of keys and values, the attention
that reads it, and attention over whole prompts.

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors are torch CUDA tensors; calls are enqueued on the current torch
stream (or `stream`). What torch can see of an argument (type, shape,
strides, device) is checked here and raises ValueError; a nonzero status of
the library raises RuntimeError. There is no fallback.
"""
from __future__ import annotations

import ctypes
import math

from . import _native
from ._native import _check, _ptr, _stream

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


_CACHE, _HEADS = ctypes.POINTER(CacheStruct), ctypes.POINTER(Heads)

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


def _dtype_code(t):
    import torch
    code = {torch.bfloat16: BF16, torch.float16: FP16}.get(t.dtype)
    if code is None:
        raise ValueError(f"tensors are bfloat16 or float16, got {t.dtype}")
    return code


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _ints(name, t, shape, device):
    """A contiguous int32 CUDA tensor of this shape."""
    import torch
    _need(t.dtype == torch.int32 and tuple(t.shape) == tuple(shape) and t.is_contiguous() and t.device == device,
          f"{name} must be a contiguous int32 tensor {tuple(shape)} on {device}, got {t.dtype} {tuple(t.shape)} on "
          f"{t.device}")
    return _ptr(t)


def _heads(name, t, like=None):
    """[tokens, heads, dim] with dim contiguous, as moe_heads_t."""
    _need(t.dim() == 3 and t.is_cuda, f"{name} must be a CUDA tensor [tokens, heads, dim]")
    if like is not None:
        _need(t.dtype == like.dtype and t.device == like.device,
              f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    ts, hs, ds = t.stride()
    # a stride along one element says nothing
    ts, hs = (ts if t.shape[0] > 1 else 0), (hs if t.shape[1] > 1 else 0)
    _need(t.shape[2] == 1 or ds == 1, f"{name}: the last dimension must be contiguous")
    _need(ts % 8 == 0 and hs % 8 == 0, f"{name}: strides must be multiples of 8 elements, got {ts} and {hs}")
    return Heads(t.data_ptr(), ts, hs)


class KVCache:
    """A handle over a paged cache whose memory is the caller's: pages
    [2 * layers, n_pages, page_size, kv_heads, head_dim], and int32 table
    [max_seqs, max_pages], length and held [max_seqs], refs [n_pages]
    (moe_kv_cache_t)."""

    def __init__(self, pages, table, length, held, refs):
        _need(pages.dim() == 5 and pages.is_contiguous() and pages.is_cuda,
              "pages must be a contiguous CUDA tensor [2 * layers, n_pages, page_size, kv_heads, head_dim]")
        _need(table.dim() == 2, "table must be [max_seqs, max_pages]")
        planes, n_pages, page_size, heads, dim = pages.shape
        max_seqs, max_pages = table.shape
        dev = pages.device
        self.pages, self.table, self.length, self.held, self.refs = pages, table, length, held, refs
        self.layers, self.device = planes // 2, dev
        self.struct = CacheStruct(pages.data_ptr(), planes, n_pages, page_size, heads, dim, _dtype_code(pages),
                                  _ints("table", table, (max_seqs, max_pages), dev).value,
                                  _ints("length", length, (max_seqs,), dev).value,
                                  _ints("held", held, (max_seqs,), dev).value,
                                  _ints("refs", refs, (n_pages,), dev).value, max_seqs, max_pages)
        self._ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, layers, n_pages, page_size, kv_heads, head_dim, max_seqs, max_pages, dtype=None, device="cuda"):
        """A fresh cache."""
        import torch
        ints = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros((2 * layers, n_pages, page_size, kv_heads, head_dim), dtype=dtype or torch.bfloat16,
                               device=device),
                   torch.full((max_seqs, max_pages), -1, **ints), torch.zeros(max_seqs, **ints),
                   torch.zeros(max_seqs, **ints), torch.zeros(n_pages, **ints))


def pages_workspace(cache: KVCache):
    """The scratch of moe_kv_extend, moe_kv_keep and moe_kv_compact."""
    import torch
    return torch.empty(load().moe_kv_workspace_size(cache._ref), dtype=torch.uint8, device=cache.device)


def moe_kv_extend(cache: KVCache, seqs, add, workspace, stream=None):
    n = seqs.numel()
    _check("moe_kv_extend",
           load().moe_kv_extend(cache._ref, _ints("seqs", seqs, (n,), cache.device),
                                _ints("add", add, (n,), cache.device), n, _ptr(workspace), workspace.numel(),
                                _stream(stream)))


def moe_kv_append(cache: KVCache, layer: int, seqs, cu, k, v, stream=None):
    n, total = seqs.numel(), k.shape[0]
    shape = (total, cache.struct.heads_kv, cache.struct.head_dim)
    _need(tuple(k.shape) == shape and tuple(v.shape) == shape, f"k and v must be {shape}")
    _check("moe_kv_append",
           load().moe_kv_append(cache._ref, layer, _ints("seqs", seqs, (n,), cache.device),
                                _ints("cu", cu, (n + 1,), cache.device), n, total,
                                ctypes.byref(_heads("k", k, cache.pages)), ctypes.byref(_heads("v", v, cache.pages)),
                                _stream(stream)))


def moe_kv_fork(cache: KVCache, src, dst, stream=None):
    n = src.numel()
    _check("moe_kv_fork", load().moe_kv_fork(cache._ref, _ints("src", src, (n,), cache.device),
                                             _ints("dst", dst, (n,), cache.device), n, _stream(stream)))


def moe_kv_truncate(cache: KVCache, seqs, new_len, stream=None):
    n = seqs.numel()
    _check("moe_kv_truncate",
           load().moe_kv_truncate(cache._ref, _ints("seqs", seqs, (n,), cache.device),
                                  _ints("new_len", new_len, (n,), cache.device), n, _stream(stream)))


def moe_kv_keep(cache: KVCache, seqs, drafted, keep, kept, workspace, stream=None):
    n = seqs.numel()
    _need(keep.dim() == 2, "keep must be [n, max_keep]")
    _check("moe_kv_keep",
           load().moe_kv_keep(cache._ref, _ints("seqs", seqs, (n,), cache.device),
                              _ints("drafted", drafted, (n,), cache.device),
                              _ints("keep", keep, (n, keep.shape[1]), cache.device), keep.shape[1],
                              _ints("kept", kept, (n,), cache.device), n, _ptr(workspace), workspace.numel(),
                              _stream(stream)))


def moe_kv_copy_pages(cache: KVCache, src, dst, stream=None):
    n = src.numel()
    _check("moe_kv_copy_pages", load().moe_kv_copy_pages(cache._ref, _ints("src", src, (n,), cache.device),
                                                         _ints("dst", dst, (n,), cache.device), n, _stream(stream)))


def moe_kv_compact(cache: KVCache, workspace, stream=None):
    _check("moe_kv_compact", load().moe_kv_compact(cache._ref, _ptr(workspace), workspace.numel(), _stream(stream)))


def moe_tree_mask(parents, cu, mask, stream=None):
    """mask [total, words] from the drafted tokens' parents [total]."""
    n, total = cu.numel() - 1, parents.numel()
    _need(mask.dim() == 2, "mask must be [total, words]")
    _check("moe_tree_mask",
           load().moe_tree_mask(_ints("parents", parents, (total,), mask.device), _ints("cu", cu, (n + 1,), mask.device),
                                n, total, _ints("mask", mask, (total, mask.shape[1]), mask.device), mask.shape[1],
                                _stream(stream)))


def _out_and_lse(q, out, lse):
    import torch
    _need(tuple(out.shape) == tuple(q.shape), f"out must be {tuple(q.shape)}")
    if lse is not None:
        _need(lse.dtype == torch.float32 and tuple(lse.shape) == tuple(q.shape[:2]) and lse.is_contiguous()
              and lse.device == q.device, f"lse must be a contiguous float32 tensor {tuple(q.shape[:2])}")
    return ctypes.byref(_heads("out", out, q)), _ptr(lse)


def moe_attention_prompt(q, k, v, cu_q, cu_k, out, lse=None, scale=None, stream=None):
    """Causal attention over packed whole prompts; scale defaults to head_dim ** -0.5."""
    n = cu_q.numel() - 1
    total_q, heads_q, dim = q.shape
    total_k, heads_kv, _ = k.shape
    _need(k.shape[2] == dim and v.shape == k.shape, "k and v must be [total_k, kv_heads, head_dim]")
    o, e = _out_and_lse(q, out, lse)
    _check("moe_attention_prompt",
           load().moe_attention_prompt(ctypes.byref(_heads("q", q)), ctypes.byref(_heads("k", k, q)),
                                       ctypes.byref(_heads("v", v, q)), _ints("cu_q", cu_q, (n + 1,), q.device),
                                       _ints("cu_k", cu_k, (n + 1,), q.device), n, total_q, total_k, heads_q, heads_kv,
                                       dim, _dtype_code(q), 1.0 / math.sqrt(dim) if scale is None else scale, o, e,
                                       _stream(stream)))


def cached_workspace(cache: KVCache, n: int, total_q: int, heads_q: int):
    """The scratch of moe_attention_cached for calls of n sequences, total_q queries."""
    import torch
    size = load().moe_attention_cached_workspace_size(cache._ref, n, total_q, heads_q)
    return torch.empty(size, dtype=torch.uint8, device=cache.device)


def moe_attention_cached(q, cache: KVCache, layer: int, seqs, cu_q, out, workspace, mask=None, lse=None, scale=None,
                         stream=None):
    """Attention of drafted tokens (or one token a sequence) over the cache;
    mask: None for a chain, else the tree's bits (moe_tree_mask). scale
    defaults to head_dim ** -0.5."""
    n = seqs.numel()
    total_q, heads_q, dim = q.shape
    _need(dim == cache.struct.head_dim, f"q must have the cache's head_dim {cache.struct.head_dim}")
    words = 0
    if mask is not None:
        _need(mask.dim() == 2, "mask must be [total_q, words]")
        words = mask.shape[1]
        mask = _ints("mask", mask, (total_q, words), cache.device)
    o, e = _out_and_lse(q, out, lse)
    _check("moe_attention_cached",
           load().moe_attention_cached(ctypes.byref(_heads("q", q, cache.pages)), cache._ref, layer,
                                       _ints("seqs", seqs, (n,), cache.device),
                                       _ints("cu_q", cu_q, (n + 1,), cache.device), n, total_q, heads_q, mask, words,
                                       1.0 / math.sqrt(dim) if scale is None else scale, o, e, _ptr(workspace),
                                       workspace.numel(), _stream(stream)))
