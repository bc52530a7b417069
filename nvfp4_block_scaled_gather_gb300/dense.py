"""ctypes binding of the dense operators of libmoe_nvfp4.so
(include/moe_dense.h): the residual stream's step between two blocks with its
norms, rows in 8-bit floating point, and their product.

Argument marshalling only, as in attention.py: tensors are torch CUDA tensors
on the current device, calls are enqueued on the current torch stream (or
`stream`), what torch can see of an argument is checked here and raises
ValueError, a nonzero status of the library raises RuntimeError. There is no
fallback.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _native
from .attention import BF16, FP16, _scratch, _stream
from ._native import _check

c_int, c_size_t, c_void_p, c_longlong = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_longlong

FP32 = 2  # MOE_FP32


class Fp8RowsStruct(ctypes.Structure):
    """moe_fp8_rows_t"""
    _fields_ = [("codes", c_void_p), ("scales", c_void_p), ("row_stride", c_longlong), ("scale_stride", c_longlong)]


# the structs as bytes, at a fifth of the time that classes take
_rows_bytes = struct.Struct("PPqq").pack
# moe_residual_norm_t: tokens, heads, dim, dtype; x; block; gate (padded to 8 bytes); residual_scale, eps, post_norm,
# padding, post_weight, pre_weight; y; normed; quantized
_norm_bytes = struct.Struct("iiii" "Pqq" "Pqq" "PqqiI" "ffiIPP" "Pqq" "Pqq").pack
_NO_PART, _NO_GATE, _NO_ROWS = (0, 0, 0), (0, 0, 0, 0), bytes(32)

_SIGS = {
    "moe_residual_norm": (c_int, [c_void_p, c_void_p]),
    "moe_fp8_quantize_rows": (c_int, [c_void_p, c_longlong, c_int, c_int, c_int, c_void_p, c_void_p]),
    "moe_fp8_gemm": (c_int, [c_void_p, c_int, c_void_p, c_int, c_int, c_void_p, c_longlong, c_int, c_void_p]),
    "moe_fp8_linear_workspace_size": (c_size_t, [c_int, c_int]),
    "moe_fp8_linear": (c_int, [c_void_p, c_longlong, c_int, c_int, c_int, c_void_p, c_int, c_void_p, c_longlong, c_int,
                               c_void_p, c_size_t, c_void_p]),
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


_FLOAT32 = torch.float32
_CODES = {torch.bfloat16: BF16, torch.float16: FP16}
_OUT_CODES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}
_MOST = 2 ** 31 - 1  # that an int of the library holds (ctypes would pass the low 32 bits on)


class Fp8Rows:
    """8-bit rows (moe_fp8_rows_t) whose memory is the caller's: codes [rows, k], float8_e4m3fn or uint8, and scales
    [rows, at least 4 * ceil(k / 512)] uint8 (e8m0: 2 ** (byte - 127)), one for each 128 values; both contiguous along
    their rows. `rows(n)` is a handle over the first n. Values may be written in place at any time; a handle whose tensors
    have moved, or are others, since it was made is refused: make a new one."""

    def __init__(self, codes, scales):
        if codes.dim() != 2 or codes.dtype not in (torch.float8_e4m3fn, torch.uint8) or not codes.is_cuda:
            raise ValueError("codes must be a float8_e4m3fn or uint8 CUDA tensor [rows, k]")
        rows, k = codes.shape
        if max(rows, k) > _MOST:
            raise ValueError(f"codes must have less than 2**31 rows and columns, got {tuple(codes.shape)}")
        if k and codes.stride(1) != 1 or rows > 1 and (codes.stride(0) % 16 or codes.stride(0) < k):
            raise ValueError(f"codes' rows must be contiguous, apart, and a multiple of 16 bytes from each other, got "
                             f"strides {codes.stride()}")
        if scales.dtype is not torch.uint8 or scales.dim() != 2 or scales.get_device() != codes.get_device():
            raise ValueError(f"scales must be a uint8 tensor [rows, scales] on {codes.device}")
        words = 4 * -(-k // 512)
        if scales.shape[0] != rows or scales.shape[1] < words:
            raise ValueError(f"scales must be [{rows}, {words} or more], got {tuple(scales.shape)}")
        if scales.shape[1] and scales.stride(1) != 1 or rows > 1 and (scales.stride(0) % 4 or scales.stride(0) < words):
            raise ValueError(f"scales' rows must be contiguous, apart, and a multiple of 4 bytes from each other, got "
                             f"strides {scales.stride()}")
        self.codes, self.scales, self.n, self.k, self.device = codes, scales, rows, k, codes.get_device()
        # (held here too: memory at an address that is still the tensors' is still theirs, whatever became of its shape)
        self.held = codes.detach(), scales.detach()
        self.at = self.codes_were_at, self.scales_were_at = codes.data_ptr(), scales.data_ptr()
        self.bytes = _rows_bytes(*self.at, codes.stride(0) if rows > 1 else 0,
                                 scales.stride(0) if rows > 1 else 0)

    # (each with what tells its address, which every call asks)
    @property
    def codes(self):
        return self._codes

    @codes.setter
    def codes(self, t):
        self._codes, self.codes_at = t, t.data_ptr

    @property
    def scales(self):
        return self._scales

    @scales.setter
    def scales(self, t):
        self._scales, self.scales_at = t, t.data_ptr

    @classmethod
    def empty(cls, rows, k, device="cuda"):
        return cls(torch.empty((rows, k), dtype=torch.float8_e4m3fn, device=device),
                   torch.empty((rows, 4 * -(-k // 512)), dtype=torch.uint8, device=device))

    def rows(self, n):
        if not 0 <= n <= self.n:
            raise ValueError(f"there are {self.n} rows, not {n}")
        return self if n == self.n else Fp8Rows(self.codes[:n], self.scales[:n])

    def dequantized(self):
        """The values that the rows stand for, fp32 (for checks: elementary torch operations)."""
        power = torch.ldexp(torch.ones((), device=self.codes.device), self.scales.int() - 127)
        power = torch.where(self.scales == 255, torch.full_like(power, float("nan")), power)
        codes = self.codes.view(torch.float8_e4m3fn).float()
        return codes * power.repeat_interleave(128, dim=1)[:, :self.k]


def _matrix(name, t, dtype, device: int):
    """[rows, k] with k contiguous: address, row stride in elements, shape."""
    shape = t.shape
    if t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} on cuda:{device}, got {t.dtype} on {t.device}")
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix, got {tuple(shape)}")
    rows, k = shape
    if rows > _MOST or k > _MOST:
        raise ValueError(f"{name} must have less than 2**31 rows and columns, got {tuple(shape)}")
    rs, ks = t.stride()
    if rows == 0:
        rs, ks = 0, 1
    elif rows == 1:
        rs = 0
    if ks != 1 and k > 1:
        raise ValueError(f"{name}: rows must be contiguous, got strides {t.stride()}")
    return t.data_ptr(), rs, rows, k


def _input16(name, t, device: int):
    dtype, shape = t.dtype, t.shape
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float16, got {dtype}")
    # (rows without gaps are the usual ones; the library minds their length)
    if len(shape) == 2 and 0 < shape[0] <= _MOST and shape[1] <= _MOST and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr(), shape[1] if shape[0] > 1 else 0, shape[0], shape[1], code
    p, rs, rows, k = _matrix(name, t, dtype, device)
    if rs % 8:
        raise ValueError(f"{name}: the row stride must be a multiple of 8 elements, got {t.stride()}")
    return p, rs, rows, k, code


def _no_handle(name, r):
    raise ValueError(f"{name} must be Fp8Rows, got {type(r).__name__}")


def _rows_of(name, r, device: int):
    if r.device != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {r.codes.device}")
    if r.codes_at() != r.codes_were_at or r.scales_at() != r.scales_were_at:
        raise ValueError(f"{name}: its tensors are not where they were when the handle was made: make a new one")
    return r.bytes


def _output(y, rows, n, device: int):
    dtype = y.dtype
    code = _OUT_CODES.get(dtype)
    if code is None:
        raise ValueError(f"y must be bfloat16, float16 or float32, got {dtype}")
    if y.shape == (rows, n) and y.is_contiguous() and y.get_device() == device:
        return y.data_ptr(), n, code
    p, rs, rows_y, n_y = _matrix("y", y, dtype, device)
    if rows_y != rows or n_y != n:
        raise ValueError(f"y must be [{rows}, {n}], got {tuple(y.shape)}")
    return p, rs, code


def moe_fp8_quantize_rows(x, out: Fp8Rows, stream=None):
    """x [rows, k], bfloat16 or float16, as 8-bit rows."""
    if not isinstance(out, Fp8Rows):
        _no_handle("out", out)
    dev = out.device
    p, rs, rows, k, code = _input16("x", x, dev)
    if (rows, k) != (out.n, out.k):
        raise ValueError(f"out must have {rows} rows of {k}, got {out.n} of {out.k}")
    status = (_LIB or load()).moe_fp8_quantize_rows(p, rs, rows, k, code, _rows_of("out", out, dev), _stream(stream, dev))
    if status:
        _check("moe_fp8_quantize_rows", status)


def moe_fp8_gemm(x: Fp8Rows, w: Fp8Rows, y, stream=None):
    """y [x's rows, w's rows] = x w^T over dequantized values, bfloat16, float16 or float32."""
    if not isinstance(w, Fp8Rows):
        _no_handle("w", w)
    dev = w.device
    if not isinstance(x, Fp8Rows):
        _no_handle("x", x)
    if x.k != w.k:
        raise ValueError(f"x and w must have rows of one length, got {x.k} and {w.k}")
    p, rs, code = _output(y, x.n, w.n, dev)
    status = (_LIB or load()).moe_fp8_gemm(_rows_of("x", x, dev), x.n, _rows_of("w", w, dev), w.n, w.k, p, rs, code,
                                           _stream(stream, dev))
    if status:
        _check("moe_fp8_gemm", status)


def linear_workspace(tokens: int, k: int, device="cuda"):
    """The scratch of moe_fp8_linear for calls of up to `tokens` rows of k."""
    size = load().moe_fp8_linear_workspace_size(tokens, k) if 0 <= tokens <= _MOST and 0 <= k <= _MOST else 0
    if size == 0:
        raise ValueError(f"no product of {tokens} rows of {k}: k must be a positive multiple of 16, both within limits")
    return torch.empty(size, dtype=torch.uint8, device=device)


def moe_fp8_linear(x, w: Fp8Rows, y, workspace, stream=None):
    """y = x w^T with x [rows, k], bfloat16 or float16, quantized on the way: moe_fp8_quantize_rows, then
    moe_fp8_gemm."""
    if not isinstance(w, Fp8Rows):
        _no_handle("w", w)
    dev = w.device
    p, rs, rows, k, code = _input16("x", x, dev)
    if k != w.k:
        raise ValueError(f"x and w must have rows of one length, got {k} and {w.k}")
    py, rsy, code_y = _output(y, rows, w.n, dev)
    ws, ws_bytes = _scratch(workspace, dev)
    status = (_LIB or load()).moe_fp8_linear(p, rs, rows, k, code, _rows_of("w", w, dev), w.n, py, rsy, code_y, ws,
                                             ws_bytes, _stream(stream, dev))
    if status:
        _check("moe_fp8_linear", status)


def _part(name, t, dtype, tokens, heads, dim, device: int):
    """[tokens, dim] or [tokens, heads, dim] with dim contiguous: address, token and head stride."""
    if t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} on cuda:{device}, got {t.dtype} on {t.device}")
    shape = t.shape
    if len(shape) == 3:
        if shape[0] != tokens or shape[1] != heads or shape[2] != dim:
            raise ValueError(f"{name} must be like x {(tokens, heads, dim)}, got {tuple(shape)}")
    elif len(shape) != 2 or heads != 1 or shape[0] != tokens or shape[1] != dim:
        raise ValueError(f"{name} must be like x {(tokens, heads, dim)}, got {tuple(shape)}")
    if t.is_contiguous():
        ts, hs = heads * dim, dim
    else:
        strides = t.stride()
        ts, hs, ds = strides if len(strides) == 3 else (strides[0], 0, strides[1])
        if ds != 1 and dim != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous, got {strides}")
    # a stride along one element says nothing
    if tokens <= 1:
        ts = 0
    if heads <= 1:
        hs = 0
    if ts % 8 or hs % 8:
        raise ValueError(f"{name}: the strides of tokens and heads must be multiples of 8 elements, got {t.stride()}")
    return t.data_ptr(), ts, hs


def _norm_weight(name, w, dim, device: int):
    if w.dtype is not _FLOAT32 or w.shape != (dim,) or not w.is_contiguous() or w.get_device() != device:
        raise ValueError(f"{name} must be a contiguous float32 tensor {(dim,)} on cuda:{device}")
    return w.data_ptr()


def _gate(g, dtype, shape, device: int):
    """A factor for each element, by broadcasting: sizes of 1 are held along. Address and strides."""
    if g.dtype is not dtype or g.get_device() != device:
        raise ValueError(f"gate must be {dtype} on cuda:{device}, got {g.dtype} on {g.device}")
    tokens, heads, dim = shape
    sizes, strides = g.shape, g.stride()
    if len(sizes) == 3:
        (t, h, d), (ts, hs, ds) = sizes, strides
    elif len(sizes) == 2 and heads == 1:
        (t, d), h, (ts, ds), hs = sizes, 1, strides, 0
    else:
        raise ValueError(f"gate must broadcast to {tuple(shape)}, got {tuple(sizes)}")
    if t != tokens and t != 1 or h != heads and h != 1 or d != dim and d != 1:
        raise ValueError(f"gate must broadcast to {tuple(shape)}, got {tuple(sizes)}")
    if t == 1:
        ts = 0
    if h == 1:
        hs = 0
    if d == 1:
        ds = 0
    if ds != 0 and ds != 1 or ds == 1 and (ts % 8 or hs % 8):
        raise ValueError(f"gate: the last dimension must be contiguous (or 1) and the other strides multiples of 8 "
                         f"elements, got {strides}")
    return g.data_ptr(), ts, hs, ds


def moe_residual_norm(x, block=None, *, y=None, normed=None, quantized: Fp8Rows = None, pre_weight=None,
                      post_norm=False, post_weight=None, gate=None, residual_scale=1.0, eps=1e-6, stream=None):
    """The residual stream takes up a block's output and is normed for the next one (moe_residual_norm_t):

      b      = norm(block) * post_weight if post_norm else block
      y      = x + residual_scale * gate * b        (x without a block)
      normed = norm(y) * pre_weight                 (quantized: the same as 8-bit rows)

    x, block, y and normed [tokens, dim], or [tokens, heads, dim] with every head normed by itself; outputs that are
    None are not written. gate broadcasts to x's shape."""
    dtype, dev, shape = x.dtype, x.get_device(), x.shape
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"x must be bfloat16 or float16, got {dtype}")
    if len(shape) == 2:
        (tokens, dim), heads = shape, 1
    elif len(shape) == 3:
        tokens, heads, dim = shape
    else:
        raise ValueError(f"x must be [tokens, dim] or [tokens, heads, dim], got {tuple(shape)}")
    if max(shape) > _MOST:
        raise ValueError(f"x must have less than 2**31 of each, got {tuple(shape)}")
    # of tensors like x without gaps (the usual ones) all is known but the address
    whole = (heads * dim if tokens > 1 else 0, dim if heads > 1 else 0)

    def part(name, t):
        if t is None:
            return _NO_PART
        if t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev:
            return (t.data_ptr(), *whole)
        return _part(name, t, dtype, tokens, heads, dim, dev)

    rows = _NO_ROWS
    if quantized is not None:
        if not isinstance(quantized, Fp8Rows):
            _no_handle("quantized", quantized)
        rows = _rows_of("quantized", quantized, dev)
        if quantized.n != tokens or quantized.k != dim or heads != 1:
            raise ValueError(f"quantized must have {tokens} rows of {dim} (of one head), got {quantized.n} of {quantized.k}")
    px = (x.data_ptr(), *whole) if x.is_contiguous() else _part("x", x, dtype, tokens, heads, dim, dev)
    args = _norm_bytes(tokens, heads, dim, code, *px, *part("block", block),
                       *(_NO_GATE if gate is None else _gate(gate, dtype, (tokens, heads, dim), dev)), 0,
                       residual_scale, eps, 1 if post_norm else 0, 0,
                       0 if post_weight is None else _norm_weight("post_weight", post_weight, dim, dev),
                       0 if pre_weight is None else _norm_weight("pre_weight", pre_weight, dim, dev),
                       *part("y", y), *part("normed", normed)) + rows
    status = (_LIB or load()).moe_residual_norm(args, _stream(stream, dev))
    if status:
        _check("moe_residual_norm", status)
