"""The dense operators' C ABI and binding without a GPU: the library exports
what the header declares, bad arguments are refused on the host before any CUDA
call. And the definitions that the GPU tests hold the kernels to."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import dense as D
from oracle import dense as OD
from tests.conftest import ROOT

INVALID, SHAPE, WORKSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def lib(native):
    return D.load()


def rows(codes=4096, scales=4096, stride=256, scale_stride=4):
    """8-bit rows at made-up aligned addresses: nothing here reaches the device."""
    return ctypes.byref(D.Fp8RowsStruct(codes, scales, stride, scale_stride))


def test_library_exports_every_declared_symbol(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_dense.h")).read(), flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", src, flags=re.M)
    assert set(names) == set(D.exported_symbols())
    for n in names:
        assert hasattr(lib, n), n


def test_quantize_refusals(lib):
    def call(x=4096, stride=256, n=4, k=256, dtype=0, out=None):
        return lib.moe_fp8_quantize_rows(x, stride, n, k, dtype, rows() if out is None else out, None)

    for bad in (dict(x=None), dict(x=4098), dict(stride=100), dict(stride=-8), dict(n=-1), dict(k=0), dict(k=-16), dict(dtype=2),
                dict(out=rows(codes=0)), dict(out=rows(scales=0)), dict(out=rows(codes=4104)), dict(out=rows(scales=4098)),
                dict(out=rows(stride=240)), dict(out=rows(stride=264)), dict(out=rows(scale_stride=0)),
                dict(out=rows(scale_stride=6)), dict(k=1024, out=rows(stride=1024))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(k=250), dict(k=8), dict(k=(1 << 20) + 16), dict(n=1 << 24)):
        assert call(**bad) == SHAPE, bad
    assert call(n=0, x=None, out=rows(codes=0)) == 0


def test_gemm_refusals(lib):
    def call(x=rows(), t=4, w=rows(), n=8, k=256, y=4096, stride=8, dtype=0):
        return lib.moe_fp8_gemm(x, t, w, n, k, y, stride, dtype, None)

    for bad in (dict(x=None), dict(w=None), dict(x=rows(codes=0)), dict(w=rows(scales=0)), dict(x=rows(stride=128)),
                dict(w=rows(stride=1 << 40)), dict(w=rows(scale_stride=2)), dict(t=-1), dict(n=-1), dict(k=0), dict(y=None),
                dict(y=4097), dict(y=4098, dtype=2), dict(stride=7), dict(stride=-8), dict(dtype=3), dict(dtype=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(k=24), dict(k=1 << 21), dict(t=1 << 24), dict(n=1 << 24)):
        assert call(**bad) == SHAPE, bad
    assert call(t=0, x=None, y=None) == 0 and call(n=0, w=None, y=None) == 0


def test_linear_refusals(lib):
    size = lib.moe_fp8_linear_workspace_size(4, 256)
    assert size >= 4 * 256 + 4 * 4
    for t, k in ((-1, 256), (4, 0), (4, 250), (4, -16), (1 << 24, 256), (4, 1 << 21)):
        assert lib.moe_fp8_linear_workspace_size(t, k) == 0
    assert lib.moe_fp8_linear_workspace_size(0, 256) > 0

    def call(x=4096, xs=256, t=4, k=256, dtype=0, w=rows(), n=8, y=4096, ys=8, y_dtype=2, ws=256, ws_bytes=size):
        return lib.moe_fp8_linear(x, xs, t, k, dtype, w, n, y, ys, y_dtype, ws, ws_bytes, None)

    for bad in (dict(x=None), dict(x=4100), dict(xs=4), dict(t=-1), dict(k=0), dict(dtype=2), dict(w=None), dict(w=rows(stride=0)),
                dict(n=-1), dict(y=None), dict(ys=7), dict(y_dtype=3), dict(ws=None), dict(ws=272)):
        assert call(**bad) == INVALID, bad
    assert call(k=264) == SHAPE
    assert call(ws_bytes=size - 1) == WORKSPACE
    assert call(t=0, x=None) == 0 and call(n=0) == 0


def norm_args(tokens=4, heads=1, dim=256, dtype=0, x=(4096, 256, 0), block=(8192, 256, 0), gate=(0, 0, 0, 0), scale=1.0, eps=1e-6,
              post=0, post_weight=0, pre_weight=0, y=(12288, 256, 0), normed=(16384, 256, 0), quantized=(0, 0, 0, 0)):
    return D._norm_bytes(tokens, heads, dim, dtype, *x, *block, *gate, 0, scale, eps, post, 0, post_weight, pre_weight, *y,
                         *normed) + D._rows_bytes(*quantized)


def test_norm_refusals(lib):
    def call(**other):
        return lib.moe_residual_norm(norm_args(**other), None)

    none = (0, 0, 0)
    for bad in (dict(tokens=-1), dict(heads=0), dict(dim=0), dict(dtype=2), dict(dtype=-1), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(scale=float("inf")), dict(scale=float("nan")), dict(post=2),
                dict(x=none), dict(x=(4100, 256, 0)), dict(x=(4096, 100, 0)), dict(x=(4096, -8, 0)),
                dict(block=none), dict(block=none, y=none, post=1), dict(block=none, y=none, gate=(4096, 0, 0, 0)),
                dict(block=(8200, 256, 0)), dict(post_weight=4096), dict(post=1, post_weight=4100), dict(pre_weight=4100),
                dict(y=none, normed=none), dict(y=(12288, 0, 0)), dict(y=(12288, 248, 0)), dict(y=(12300, 256, 0)),
                dict(normed=(12288, 256, 0)), dict(normed=(16384, 128, 0)), dict(heads=2, x=(4096, 512, 256)),
                dict(gate=(4098, 0, 0, 1)), dict(gate=(4096, 4, 0, 1)), dict(gate=(4097, 4, 0, 0)), dict(gate=(4096, -1, 0, 0)),
                dict(gate=(4096, 0, 0, 2)), dict(quantized=(4096, 0, 256, 4)), dict(quantized=(4096, 4096, 240, 4))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dim=252), dict(dim=16392), dict(tokens=1 << 20, heads=1 << 12), dict(dim=264, quantized=(4096, 4096, 272, 4)),
                dict(heads=2, quantized=(4096, 4096, 256, 4))):
        assert call(**bad) == SHAPE, bad
    assert lib.moe_residual_norm(None, None) == INVALID
    assert call(tokens=0) == 0


def test_binding_refuses_what_torch_can_see():
    codes, scales = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8)
    with pytest.raises(ValueError, match="codes must be"):
        D.Fp8Rows(codes, scales)  # not on a GPU
    with pytest.raises(ValueError, match="must be bfloat16 or float16"):
        D.moe_residual_norm(torch.zeros((2, 8)))
    for x, block in (((2, 8), (2, 16)), ((2, 8), (3, 8)), ((2, 2, 8), (2, 16)), ((2, 8), (2, 2, 8)), ((2, 8), (8,))):
        with pytest.raises(ValueError, match="like x"):
            D.moe_residual_norm(torch.zeros(x, dtype=torch.bfloat16), torch.zeros(block, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="tokens, dim"):
        D.moe_residual_norm(torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        D.moe_residual_norm(torch.zeros((8, 16), dtype=torch.bfloat16)[:, ::2])
    with pytest.raises(ValueError, match="multiples of 8"):
        D.moe_residual_norm(torch.zeros((8, 12), dtype=torch.bfloat16)[:, :8])
    with pytest.raises(ValueError, match="post_weight must be"):
        D._norm_weight("post_weight", torch.zeros(8, dtype=torch.bfloat16), 8, -1)
    x = torch.zeros((2, 3, 8), dtype=torch.bfloat16)
    for gate, text in ((torch.zeros((2, 3, 4), dtype=torch.bfloat16), "broadcast"), (torch.zeros((2, 8), dtype=torch.bfloat16), "broadcast"),
                       (x.float(), "must be torch.bfloat16"), (x[:, :, ::2].expand(2, 3, 4), "broadcast"),
                       (torch.zeros((2, 3, 16), dtype=torch.bfloat16)[..., ::2], "contiguous"),
                       (torch.zeros((2, 3, 9), dtype=torch.bfloat16)[..., :8], "multiples of 8")):
        with pytest.raises(ValueError, match=text):
            D._gate(gate, torch.bfloat16, (2, 3, 8), -1)
    strides = [D._gate(g, torch.bfloat16, s, -1)[1] for g, s in (
        (torch.zeros((2, 1, 1), dtype=torch.bfloat16), (2, 3, 8)), (torch.zeros((1, 1, 8), dtype=torch.bfloat16), (2, 3, 8)),
        (torch.zeros((2, 8), dtype=torch.bfloat16), (2, 1, 8)))]
    assert strides == [1, 0, 8]
    with pytest.raises(ValueError, match="less than 2"):
        D._matrix("x", torch.zeros((1, 8), dtype=torch.bfloat16).expand(2 ** 31, 8), torch.bfloat16, -1)
    with pytest.raises(ValueError, match="contiguous"):
        D._matrix("x", torch.zeros((4, 8), dtype=torch.bfloat16).T, torch.bfloat16, -1)


def test_definition_of_8_bit_rows():
    assert OD.TABLE[[0, 1, 7, 8, 15, 0x77, 0x7E]].tolist() == [0, 2 ** -9, 7 * 2 ** -9, 2 ** -6, 15 * 2 ** -9, 240, 448]
    half = (OD.TABLE[1:] + OD.TABLE[:-1]) / 2
    assert (OD.e4m3_encode(half) % 2 == 0).all()  # ties to even
    for sign in (1, -1):
        assert np.array_equal(OD.e4m3_decode(OD.e4m3_encode(sign * OD.TABLE[1:])), sign * OD.TABLE[1:])
    want = torch.from_numpy(np.random.RandomState(0).randn(4000) * 40).float()
    assert np.array_equal(OD.e4m3_encode(want.double().numpy()), want.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert OD.scale_byte(448.0) == 127 and OD.scale_byte(np.nextafter(448, 449)) == 128 and OD.scale_byte(224.0) == 126
    assert OD.scale_byte(0.0) == 0 and OD.scale_byte(2.0 ** -140) == 0
    codes, scales = OD.quantize_rows(np.array([[1.0] * 128 + [500.0] * 2, [np.inf, 3.0, np.nan] + [0.0] * 127]))
    assert scales[:, :2].tolist() == [[119, 128], [120, 0]] and (scales[:, 2:] == 127).all()
    assert codes[1, :3].tolist() == [0x7F, 0x7C, 0x7F]
    assert OD.dequantize(codes, scales)[0, [0, 127, 128]].tolist() == [1.0, 1.0, 512.0]  # 250 is nearer to 256 than to 240


def test_definition_of_the_residual_step():
    x, b = np.array([[3.0, 4.0]]), np.array([[1.0, 7.0]])
    y, n, _ = OD.residual_norm(x, b, gate=np.array([[2.0]]), residual_scale=0.5, eps=1e-12, post_norm=True,
                               post_weight=np.array([1.0, 2.0]), pre_weight=np.array([1.0, -1.0]))
    want = np.array([3 + 1 / 5, 4 + 2 * 7 / 5])
    assert np.allclose(y, want) and np.allclose(n, want / np.sqrt((want ** 2).mean()) * [1, -1])
    assert np.array_equal(OD.residual_norm(x)[0], x)
