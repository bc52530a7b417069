"""The dense operators on the GPU against their definitions in 64 bits."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import _native as N
from nvfp4_block_scaled_gather_gb300 import dense as D
from oracle import dense as OD

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}   # half a step, relative
LEAST = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}               # half a step of the smallest values


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(DTYPES[dtype])


def f64(t):
    return t.double().cpu().numpy()


def guarded(rows, n, dtype, stride=None, value=7.0):
    """A matrix inside a larger one, and a check that nothing around it was written."""
    stride = stride or n + 24
    whole = torch.full((rows + 6, stride), value, dtype=DTYPES[dtype], device="cuda")
    inside = whole[3:3 + rows, 8:8 + n]

    def untouched():
        whole[3:3 + rows, 8:8 + n] = value
        return bool((whole == value).all())

    return inside, untouched


# ------------------------------------------------------------------------------------------------ 8-bit rows

def quantize(x, out=None):
    out = out or D.Fp8Rows.empty(*x.shape)
    D.moe_fp8_quantize_rows(x, out)
    torch.cuda.synchronize()
    assert N.check_status() == 0
    return out


def bits(rows):
    return rows.codes.view(torch.uint8).cpu().numpy(), rows.scales.cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,k", [(1, 16), (3, 112), (2, 128), (5, 144), (1, 512), (4, 528), (130, 1040), (7, 4096)])
def test_quantized_rows_are_the_definitions(cuda, rows, k, dtype):
    x = normal((rows, k), dtype, rows + k) * torch.exp2(torch.arange(rows, device="cuda") % 23 - 11.0)[:, None].to(DTYPES[dtype])
    x[0, :16] = torch.tensor([0.0, -0.0, 1, -1, 2, 3, 448, 447, 1e-3, -1e-3, 2.0 ** -9, 2.0 ** -10, 2.0 ** -11, -2.0 ** -14, 17, 19])
    for got, want in zip(bits(quantize(x)), OD.quantize_rows(f64(x))):
        assert np.array_equal(got, want)


def test_every_bf16_maximum_and_a_ladder_below_it(cuda):
    """Each finite bf16 magnitude as a block's maximum, with a ladder of values below it."""
    size = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros((len(size), 128), dtype=torch.bfloat16)
    x[:, 0] = size
    ladder = torch.linspace(-1, 1, 127, dtype=torch.float64) ** 5
    x[:, 1:] = (size.double()[:, None] * ladder).bfloat16()
    x = x.cuda()
    codes, scales = bits(quantize(x))
    v = f64(x)
    want = np.array([OD.scale_byte(a) for a in f64(size)], np.uint8)
    assert np.array_equal(scales[:, 0], want) and (scales[:, 1:] == 127).all()
    assert np.array_equal(codes, OD.e4m3_encode(v / 2.0 ** (want[:, None].astype(float) - 127)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_infinities_and_nan_are_nan_codes_and_no_others(cuda, dtype):
    x = normal((6, 400), dtype, 5)
    for r, v in enumerate((np.inf, -np.inf, np.nan)):
        x[r, 130] = v
    x[3] = np.nan
    x[4, :128] = 0.0
    got = quantize(x)
    for g, want in zip(bits(got), OD.quantize_rows(f64(x))):
        assert np.array_equal(g, want)
    assert torch.isnan(got.dequantized()).sum(1).tolist() == [1, 1, 1, 400, 0, 0]


def test_quantizing_strided_rows_into_strided_rows(cuda):
    x = normal((9, 1000), "bf16", 6)[:, 8:8 + 656]
    codes = torch.full((11, 704), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((11, 16), 77, dtype=torch.uint8, device="cuda")
    quantize(x, D.Fp8Rows(codes[1:10, 16:16 + 656], scales[1:10, :8]))
    want = OD.quantize_rows(f64(x))
    assert np.array_equal(codes[1:10, 16:672].cpu().numpy(), want[0]) and np.array_equal(scales[1:10, :8].cpu().numpy(), want[1])
    codes[1:10, 16:672] = 77
    scales[1:10, :8] = 77
    assert (codes == 77).all() and (scales == 77).all()


# ------------------------------------------------------------------------------------------------ products

def whole_rows(rows, k, seed, most=4):
    """8-bit rows of small whole numbers under scales of 1/2, 1 and 2: every sum of products is exact in fp32."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    values = torch.randint(-most, most + 1, (rows, k), device="cuda", generator=g).float()
    scales = torch.randint(126, 129, (rows, 4 * -(-k // 512)), device="cuda", generator=g, dtype=torch.uint8)
    return D.Fp8Rows(values.to(torch.float8_e4m3fn), scales)


def gemm(x, w, dtype="fp32"):
    y, untouched = guarded(x.n, w.n, dtype)
    D.moe_fp8_gemm(x, w, y)
    torch.cuda.synchronize()
    assert N.check_status() == 0
    got = y.clone()
    assert untouched()
    return got


TOKENS = [1, 2, 7, 16, 17, 33, 64, 100, 129, 240, 241, 300, 511, 1000]


@pytest.mark.parametrize("t", TOKENS)
@pytest.mark.parametrize("n,k", [(128, 128), (1, 16), (96, 528), (300, 1040), (129, 4112)])
def test_products_of_whole_numbers_are_exact(cuda, t, n, k):
    """At most 4112 products of at most 4 * 4 * 4, multiples of 1/4: below 2^20 quarters, exact in any order."""
    x, w = whole_rows(t, k, t), whole_rows(n, k, n + 1)
    want = (x.dequantized().double() @ w.dequantized().double().T).float()
    assert torch.equal(gemm(x, w), want)


@pytest.mark.parametrize("t,n,k", [(1, 5000, 256), (20, 2500, 9216), (3, 40000, 16), (64, 1000, 16384), (1500, 1100, 512), (4097, 257, 144),
                                   (700, 2000, 20480), (2, 64, 65536)])
def test_larger_products_of_whole_numbers_are_exact(cuda, t, n, k):
    x, w = whole_rows(t, k, t, 2), whole_rows(n, k, n + 1, 2)
    want = (x.dequantized().double() @ w.dequantized().double().T).float()
    assert torch.equal(gemm(x, w), want)


def products_hold(got, x, w, dtype):
    """Every product and every addition loses a unit of fp32 at most of the sum of magnitudes, whatever their order: K +
    K / 16 + 8 times 2^-24 of it; then the result's own rounding."""
    xs, ws = x.dequantized().double(), w.dequantized().double()
    want, size = xs @ ws.T, xs.abs() @ ws.abs().T
    slack = (x.k + x.k / 16 + 8) * 2.0 ** -24 * size
    assert bool(((got.double() - want).abs() <= slack * 2 + HALF[dtype] * want.abs() + LEAST[dtype]).all())
    # and together they do far better: the framework's bound of 1e-5 on products, with the rounding beside it
    off = float((got.double() - want).norm() / want.norm())
    assert off <= 1e-5 + HALF[dtype], off


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("t,n,k", [(1, 640, 4096), (5, 384, 2064), (16, 200, 8192), (50, 1000, 1024), (333, 1000, 2064), (800, 700, 4096)])
def test_products_of_rows_against_64_bits(cuda, t, n, k, dtype):
    x, w = quantize(normal((t, k), "bf16", t)), quantize(normal((n, k), "bf16", n, k ** -0.5))
    products_hold(gemm(x, w, dtype), x, w, dtype)


def test_scales_reach_over_the_whole_range(cuda):
    """Scales of x and w whose product stays near 1 while each goes to its ends; 2^-127 to 2^120."""
    k = 512
    x, w = whole_rows(24, k, 1, 1), whole_rows(130, k, 2, 1)
    e = torch.tensor([[7, 100, 127, 154], [0, 20, 200, 247]], dtype=torch.uint8, device="cuda")
    for a in (0, 1):
        x.scales[:] = e[a]
        w.scales[:] = 254 - e[a]
        want = (x.dequantized().double() @ w.dequantized().double().T).float()
        assert torch.equal(gemm(x, w), want)


def test_a_rows_bits_do_not_depend_on_the_other_rows(cuda):
    for n, k in ((640, 4096), (200, 9216), (1100, 528)):
        x, w = quantize(normal((600, k), "bf16", 1)), quantize(normal((n, k), "bf16", 2, k ** -0.5))
        whole = gemm(x, w)
        for t in (1, 3, 16, 40, 64, 65, 128, 200, 256, 500):
            assert torch.equal(gemm(x.rows(t), w), whole[:t]), (n, k, t)
        for a, b in ((599, 600), (100, 117), (300, 433)):
            assert torch.equal(gemm(D.Fp8Rows(x.codes[a:b], x.scales[a:b]), w), whole[a:b])
        some = D.Fp8Rows(w.codes[128:190], w.scales[128:190])  # and a column's not on the other columns
        assert torch.equal(gemm(x.rows(70), some), whole[:70, 128:190])


@pytest.mark.parametrize("t", [1, 40, 300])
def test_nan_rows_reach_their_own_results_alone(cuda, t):
    """Codes for NaN and scales of 255; and what stands between rows, behind K, and behind the last row is not read."""
    n, k = 200, 656
    wide = [torch.full((rows + 4, 704), 0x7F, dtype=torch.uint8, device="cuda") for rows in (t, n)]
    scales = [torch.full((rows + 4, 12), 255, dtype=torch.uint8, device="cuda") for rows in (t, n)]
    x, w = whole_rows(t, k, 1), whole_rows(n, k, 2)
    for m, c, s in ((x, wide[0], scales[0]), (w, wide[1], scales[1])):
        c[2:-2, 16:16 + k] = m.codes.view(torch.uint8)
        s[2:-2, :6] = m.scales[:, :6]
    xs = D.Fp8Rows(wide[0][2:-2, 16:16 + k], scales[0][2:-2, :8])
    ws = D.Fp8Rows(wide[1][2:-2, 16:16 + k], scales[1][2:-2, :8])
    want = (x.dequantized().double() @ w.dequantized().double().T).float()
    assert torch.equal(gemm(xs, ws), want)
    wide[1][2 + 77, 16 + 655] = 0x7F
    scales[1][2 + 130, 0] = 255
    wide[0][2 + t // 2, 16] = 0xFF
    got = gemm(xs, ws)
    bad = torch.zeros((t, n), dtype=torch.bool, device="cuda")
    bad[:, [77, 130]] = True
    bad[t // 2] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


def test_results_past_the_types_largest_are_infinite(cuda):
    x, w = whole_rows(3, 128, 1), whole_rows(8, 128, 2)
    x.codes[:] = torch.full((3, 128), 448.0, device="cuda").to(torch.float8_e4m3fn)
    w.codes[:] = x.codes[:1]
    x.scales[:], w.scales[:] = 127, 127
    assert torch.isinf(gemm(x, w, "fp16")).all()                       # 128 * 448^2 > 65504
    assert (gemm(x, w) == 128 * 448.0 ** 2).all()
    x.scales[:], w.scales[:] = 247, 247
    assert torch.isinf(gemm(x, w)).all() and torch.isinf(gemm(x, w, "bf16")).all()


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32")])
@pytest.mark.parametrize("t,n,k", [(1, 300, 1040), (12, 500, 4096), (16, 257, 80), (17, 384, 2048), (25, 640, 9216), (32, 20000, 1024), (29, 130, 20480), (9, 25000, 528), (64, 1000, 512), (70, 100, 4096), (200, 640, 4112), (1000, 256, 528)])
def test_linear_is_quantizing_then_the_product(cuda, t, n, k, dtype, out):
    x = normal((t, k + 24), dtype, t)[:, 8:8 + k]
    w = quantize(normal((n, k), "bf16", n, k ** -0.5))
    want = gemm(quantize(x), w, out)
    y, untouched = guarded(t, n, out)
    ws = torch.full((D.load().moe_fp8_linear_workspace_size(t, k) + 256,), 255, dtype=torch.uint8, device="cuda")
    D.moe_fp8_linear(x, w, y, ws[:-256])
    torch.cuda.synchronize()
    assert N.check_status() == 0 and torch.equal(y, want) and untouched() and (ws[-256:] == 255).all()


@pytest.mark.parametrize("t", [1, 30])
def test_linear_of_rows_with_infinities(cuda, t):
    x, w = normal((t, 272), "bf16", 3), quantize(normal((100, 272), "bf16", 4))
    x[t // 2, 200] = np.inf
    y = torch.empty((t, 100), device="cuda")
    D.moe_fp8_linear(x, w, y, D.linear_workspace(t, 272))
    assert torch.isnan(y[t // 2]).all() and torch.isfinite(y).sum() == (t - 1) * 100
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(gemm(quantize(x), w)))


def test_nothing_to_do(cuda):
    w = quantize(normal((40, 64), "bf16", 1))
    empty = D.Fp8Rows.empty(0, 64)
    D.moe_fp8_quantize_rows(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), empty)
    D.moe_fp8_gemm(empty, w, torch.empty((0, 40), device="cuda"))
    D.moe_fp8_gemm(w, empty, torch.empty((40, 0), device="cuda"))
    D.moe_fp8_linear(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w, torch.empty((0, 40), device="cuda"),
                     D.linear_workspace(0, 64))
    D.moe_residual_norm(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert N.check_status() == 0


def test_no_tokens_of_everything(cuda):
    """Tensors without elements have no address."""
    x, ones = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    D.moe_residual_norm(x, x.clone(), y=x.clone(), normed=x.clone(), quantized=D.Fp8Rows.empty(0, 64), pre_weight=ones,
                        post_norm=True, post_weight=ones, gate=torch.ones((1, 64), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert N.check_status() == 0


FIRST_CALLS = """
import torch
from nvfp4_block_scaled_gather_gb300 import _native as N, dense as D
rows = [torch.randn((t, 1040), device="cuda").bfloat16() for t in (1, 20, 300)]
w, ones = D.Fp8Rows.empty(384, 1040), torch.ones(1040, device="cuda")
w.codes.view(torch.uint8).copy_(torch.randint(0, 120, (384, 1040), device="cuda"))
w.scales.fill_(120)
def outputs():
    return [(torch.zeros_like(x), D.Fp8Rows.empty(*x.shape), torch.zeros((x.shape[0], 384), device="cuda"),
             torch.zeros((x.shape[0], 384), device="cuda"), D.linear_workspace(*x.shape)) for x in rows]
def calls(outs):
    for x, (n, q, y, z, ws) in zip(rows, outs):
        D.moe_residual_norm(x, x, y=n, quantized=q, pre_weight=ones, post_norm=True)
        D.moe_fp8_gemm(q, w, y)
        D.moe_fp8_linear(x, w, z, ws)
captured, eager = outputs(), outputs()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls(captured)
graph.replay()
calls(eager)
torch.cuda.synchronize()
assert N.check_status() == 0
for a, b in zip(captured, eager):
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]) and torch.equal(a[3], b[3]) and a[2].any() and a[3].any()
"""


def test_a_process_whose_first_calls_are_captured(cuda):
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_a_graph_replays_products_on_new_inputs_and_another_stream(cuda):
    """moe_fp8_linear at several sizes and the norm, captured; replayed with other inputs; beside it the same calls on
    another stream with workspaces of their own."""
    w = quantize(normal((384, 1040), "bf16", 1, 0.03))
    xs = [normal((t, 1040), "bf16", t) for t in (1, 20, 300)]
    ys = [torch.zeros((x.shape[0], 384), dtype=torch.bfloat16, device="cuda") for x in xs]
    ws = [D.linear_workspace(*x.shape) for x in xs]
    normed = [torch.zeros_like(x) for x in xs]

    def step(xs, ys, ws, normed):
        for x, y, s, n in zip(xs, ys, ws, normed):
            D.moe_residual_norm(x, normed=n)
            D.moe_fp8_linear(n, w, y, s)

    step(xs, ys, ws, normed)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(xs, ys, ws, normed)
    for seed in (5, 6):
        for x in xs:
            x.copy_(normal(x.shape, "bf16", seed + x.shape[0]))
        other = [[torch.zeros_like(t) for t in ts] for ts in (ys, ws, normed)]
        side = torch.cuda.Stream()
        torch.cuda.synchronize()  # (the side stream's tensors are made on this one)
        graph.replay()
        with torch.cuda.stream(side):
            step(xs, *other)
        torch.cuda.synchronize()
        assert N.check_status() == 0
        for x, y, n, y2 in zip(xs, ys, normed, other[0]):
            assert torch.equal(y, y2) and torch.equal(y, gemm(quantize(n), w, "bf16"))


def test_weights_written_by_the_call_before_the_product(cuda):
    """Nothing of w is used before the call that writes it is done: quantized weights and their product back to back."""
    for t in (1, 60, 500):
        x = quantize(normal((t, 2048), "bf16", 1))
        raw = [normal((1000, 2048), "bf16", s, 0.02) for s in range(6)]
        want = [gemm(x, quantize(r)) for r in raw]
        w, ys = D.Fp8Rows.empty(1000, 2048), [torch.zeros((t, 1000), device="cuda") for _ in raw]
        for r, y in zip(raw, ys):
            D.moe_fp8_quantize_rows(r, w)
            D.moe_fp8_gemm(x, w, y)
        for a, b in zip(ys, want):
            assert torch.equal(a, b)
        step = torch.zeros_like(raw[0])
        ys = [torch.zeros((t, 1000), device="cuda") for _ in raw]
        for r, y in zip(raw, ys):  # rows of the norm as the second operand
            D.moe_residual_norm(r, quantized=w, normed=step)
            D.moe_fp8_gemm(x, w, y)
        torch.cuda.synchronize()
        for r, y in zip(raw, ys):
            D.moe_residual_norm(r, quantized=w)
            assert torch.equal(y, gemm(x, w))


# ------------------------------------------------------------------------------------------------ norms

def gate_of(kind, t, h, d, dtype, seed):
    shape = {"none": None, "token": (t, h, 1), "head": (1, h, 1), "channel": (1, 1, d), "element": (t, h, d)}[kind]
    return None if shape is None else torch.sigmoid(normal(shape, "fp32", seed)).to(DTYPES[dtype])


def norm_holds(x, block, kw, dtype, y, normed, rows=None):
    """The sums of squares are within 2^-17 of themselves (at most 128 additions deep, 64 terms a thread among them), the
    norms within half of that, and a few operations on top: 2^-17 of the magnitudes that each value is the sum of. Then
    the type's rounding."""
    arrays = {n: f64(v) if torch.is_tensor(v) else v for n, v in kw.items() if v is not None}
    wy, wn, size = OD.residual_norm(f64(x), None if block is None else f64(block), **arrays)
    slack = 2.0 ** -17 * size
    if y is not None:
        assert (np.abs(f64(y) - wy) <= slack + HALF[dtype] * (np.abs(wy) + slack) + LEAST[dtype]).all()
    factor = np.abs(kw["pre_weight"].double().cpu().numpy()) if kw.get("pre_weight") is not None else 1.0
    rms = np.sqrt((wy ** 2).mean(-1, keepdims=True) + kw["eps"])
    off = factor * slack / rms + 2.0 ** -17 * np.abs(wn)
    if normed is not None:
        assert (np.abs(f64(normed) - wn) <= off + HALF[dtype] * (np.abs(wn) + off) + LEAST[dtype]).all()
    if rows is not None:
        flat, off = wn.reshape(wn.shape[0], -1), np.broadcast_to(off, wn.shape).reshape(wn.shape[0], -1)
        codes, scales = bits(rows)
        k = flat.shape[1]
        for b in range(-(-k // 128)):
            most = np.abs(flat[:, b * 128:(b + 1) * 128]).max(1)
            s = 2.0 ** (scales[:, b].astype(float) - 127)
            assert (most <= 448 * s * (1 + 2.0 ** -12)).all()
            assert ((most > 224 * s * (1 - 2.0 ** -12)) | (scales[:, b] == 0)).all()
        assert (scales[:, -(-k // 128):] == 127).all()
        power = np.repeat(2.0 ** (scales.astype(float) - 127), 128, axis=1)[:, :k]
        assert (np.abs(OD.e4m3_decode(codes) * power - flat) <= off + 2.0 ** -4 * (np.abs(flat) + off) + 2.0 ** -10 * power).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("t,h,d", [(1, 1, 8), (5, 1, 64), (3, 7, 72), (33, 5, 128), (2, 1, 136), (9, 3, 256), (4, 1, 264), (3, 1, 512), (2, 2, 520),
                                   (1, 1, 1024), (17, 1, 2184), (1, 1, 4096), (300, 1, 4096), (3, 1, 7168), (2, 1, 8192), (3, 1, 8200), (2, 1, 16384)])
@pytest.mark.parametrize("gate,post", [("none", True), ("channel", False), ("token", True), ("element", True), ("head", False)])
def test_the_residual_step(cuda, t, h, d, dtype, gate, post):
    seed = t + h + d
    x, b = normal((t, h, d), dtype, seed, 3.0), normal((t, h, d), dtype, seed + 1)
    kw = dict(pre_weight=1 + 0.2 * normal((d,), "fp32", seed + 2), post_norm=post, gate=gate_of(gate, t, h, d, dtype, seed + 3),
              post_weight=normal((d,), "fp32", seed + 4) if post and gate != "token" else None, residual_scale=0.37, eps=1e-5)
    whole = torch.full((2, t + 2, h, d), 7.0, dtype=x.dtype, device="cuda")
    y, n = whole[0, 1:-1], whole[1, 1:-1]
    rows = D.Fp8Rows.empty(t, d) if h == 1 and d % 16 == 0 else None
    D.moe_residual_norm(x, b, y=y, normed=n, quantized=rows, **kw)
    torch.cuda.synchronize()
    norm_holds(x, b, kw, dtype, y, n, rows)
    got = whole.clone()
    assert (whole[:, 0] == 7).all() and (whole[:, -1] == 7).all()
    # each output by itself, and over the inputs: the same bits
    D.moe_residual_norm(x, b, y=x, **kw)
    assert torch.equal(x, got[0, 1:-1])
    x = normal((t, h, d), dtype, seed, 3.0)
    D.moe_residual_norm(x, b, normed=b, y=x, **kw)
    assert torch.equal(b, got[1, 1:-1]) and torch.equal(x, got[0, 1:-1])
    x, b = normal((t, h, d), dtype, seed, 3.0), normal((t, h, d), dtype, seed + 1)
    if rows is not None:
        alone = D.Fp8Rows.empty(t, d)
        D.moe_residual_norm(x, b, quantized=alone, **kw)
        assert torch.equal(alone.codes.view(torch.uint8), rows.codes.view(torch.uint8)) and torch.equal(alone.scales, rows.scales)
    if t > 1:  # a row does not depend on the others
        kw1 = {**kw, "gate": kw["gate"][t - 1:] if gate in ("token", "element") else kw["gate"]}
        one = torch.empty((1, h, d), dtype=x.dtype, device="cuda")
        D.moe_residual_norm(x[t - 1:], b[t - 1:], normed=one, **kw1)
        assert torch.equal(one, got[1, t:t + 1])
    assert N.check_status() == 0


@pytest.mark.parametrize("t,h,d", [(3001, 1, 264), (911, 1, 512), (700, 1, 776), (1300, 1, 1024), (333, 3, 2048), (40, 19, 2184), (611, 1, 3840),
                                   (460, 1, 4096), (320, 1, 5120), (170, 1, 7168), (305, 1, 8192), (330, 1, 8200), (160, 1, 14080),
                                   (155, 1, 14088), (310, 1, 16384)])
@pytest.mark.parametrize("dtype,gate,post", [("bf16", "none", True), ("fp16", "channel", False), ("fp16", "token", True), ("bf16", "element", True),
                                             ("bf16", "head", False)])
def test_the_residual_step_of_many_rows(cuda, t, h, d, dtype, gate, post):
    """More rows than run at one time: groups of threads, or CTAs, go from row to row."""
    test_the_residual_step(cuda, t, h, d, dtype, gate, post)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_heads_within_wider_rows(cuda, dtype):
    """Queries and keys of one product's rows, normed in place; the values behind them stay."""
    rows = normal((37, 14 * 64), dtype, 3)
    before = rows.clone()
    heads = rows.view(37, 14, 64)[:, :10]
    w = normal((64,), "fp32", 4)
    D.moe_residual_norm(heads, normed=heads, pre_weight=w, eps=1e-6)
    norm_holds(before.view(37, 14, 64)[:, :10], None, dict(pre_weight=w, eps=1e-6), dtype, None, heads)
    assert torch.equal(rows[:, 640:], before[:, 640:])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("t,h,d", [(700, 14, 64), (2100, 10, 64), (1001, 12, 72), (811, 9, 128), (2011, 5, 128), (613, 5, 200), (1300, 4, 256)])
def test_many_heads_within_wider_rows(cuda, t, h, d, dtype):
    """Two or four rows of a thread at a time; the values behind the heads stay."""
    rows = normal((t, (h + 2) * d), dtype, t)
    before = rows.clone()
    heads = rows.view(t, h + 2, d)[:, :h]
    w = normal((d,), "fp32", 4)
    D.moe_residual_norm(heads, normed=heads, pre_weight=w, eps=1e-6)
    norm_holds(before.view(t, h + 2, d)[:, :h], None, dict(pre_weight=w, eps=1e-6), dtype, None, heads)
    assert torch.equal(rows[:, h * d:], before[:, h * d:]) and N.check_status() == 0


@pytest.mark.parametrize("t,h,d,gate", [(30011, 4, 8, "token"), (60013, 1, 64, "channel"), (9001, 7, 128, "head"), (30011, 1, 136, "element"),
                                        (40009, 1, 256, "none")])
def test_the_residual_step_of_many_short_rows(cuda, t, h, d, gate):
    test_the_residual_step(cuda, t, h, d, "bf16", gate, True)


def test_rows_held_along_and_gates_held_along(cuda):
    """One row for all tokens as x (stride 0), a gate of one number for all."""
    x = normal((1, 1, 256), "bf16", 1).expand(5, 3, 256)
    b, g = normal((5, 3, 256), "bf16", 2), normal((1, 1, 1), "bf16", 3)
    y = torch.empty((5, 3, 256), dtype=torch.bfloat16, device="cuda")
    kw = dict(gate=g, eps=1e-6, residual_scale=2.0)
    D.moe_residual_norm(x, b, y=y, **kw)
    norm_holds(x, b, kw, "bf16", y, None)


def test_zero_rows_and_rows_that_are_not_finite(cuda):
    x, b = normal((6, 512), "bf16", 1), normal((6, 512), "bf16", 2)
    x[1] = 0
    b[1] = 0
    x[2, 7], b[3, 9], x[4, 500] = np.inf, np.nan, -np.inf
    y, n, rows = torch.empty_like(x), torch.empty_like(x), D.Fp8Rows.empty(6, 512)
    D.moe_residual_norm(x, b, y=y, normed=n, quantized=rows, post_norm=True)
    torch.cuda.synchronize()
    kw = dict(post_norm=True, eps=1e-6)
    fine = [0, 1, 5]
    some = D.Fp8Rows(rows.codes[fine].contiguous(), rows.scales[fine].contiguous())
    norm_holds(x[fine][:, None], b[fine][:, None], kw, "bf16", y[fine][:, None], n[fine][:, None], some)
    assert (y[1] == 0).all() and (n[1] == 0).all() and (rows.scales[1] == 0).all()
    # an infinity's row has an infinite sum of squares: 0 elsewhere, NaN at its place; a NaN takes its whole row
    for r, at in ((2, 7), (4, 500)):
        assert torch.isinf(y[r, at]) and torch.isfinite(y[r]).sum() == 511
        assert torch.isnan(n[r, at]) and (n[r] == 0).sum() == 511 and torch.isnan(rows.dequantized()[r]).sum() == 1
    assert torch.isnan(y[3]).all() and torch.isnan(n[3]).all() and torch.isnan(rows.dequantized()[3]).all()


def test_the_norm_into_a_product(cuda):
    """The stream's step with 8-bit rows, then the product: what the two calls give apart."""
    for t, d, n in ((1, 2048, 300), (40, 4096, 512), (400, 1040, 700)):
        x, b = normal((t, d), "bf16", t), normal((t, d), "bf16", d)
        w = quantize(normal((n, d), "bf16", n, d ** -0.5))
        rows, y = D.Fp8Rows.empty(t, d), torch.empty_like(x)
        out = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
        for _ in range(3):
            rows.codes.view(torch.uint8).fill_(0x7F)
            D.moe_residual_norm(x, b, y=y, quantized=rows, post_norm=True)
            D.moe_fp8_gemm(rows, w, out)
        torch.cuda.synchronize()
        products_hold(out, rows, w, "bf16")
        norm_holds(x[:, None], b[:, None], dict(post_norm=True, eps=1e-6), "bf16", y[:, None], None, rows)


def test_binding_refusals(cuda):
    x, w = normal((4, 64), "bf16", 1), quantize(normal((8, 64), "bf16", 2))
    ws = D.linear_workspace(4, 64)
    y = torch.empty((4, 8), device="cuda")
    for call in (lambda: D.moe_fp8_linear(x[:, :48], w, y, ws), lambda: D.moe_fp8_linear(x.float(), w, y, ws),
                 lambda: D.moe_fp8_linear(x, w, y[:3], ws), lambda: D.moe_fp8_linear(x, w, y.double(), ws),
                 lambda: D.moe_fp8_linear(x, w, y.cpu(), ws), lambda: D.moe_fp8_linear(x, w, y, ws.float()),
                 lambda: D.moe_fp8_linear(normal((4, 68), "bf16", 1)[:, :64], w, y, ws), lambda: D.moe_fp8_gemm(w, quantize(x[:, :48]), y),
                 lambda: D.moe_fp8_gemm(w, w, y), lambda: D.moe_fp8_quantize_rows(x, w), lambda: D.linear_workspace(4, 40),
                 lambda: D.moe_residual_norm(x, x[:3], y=x), lambda: D.moe_residual_norm(x, normed=x.half()),
                 lambda: D.moe_residual_norm(x, quantized=w), lambda: D.moe_residual_norm(x, x, y=x, gate=x[:, :5]),
                 lambda: D.moe_residual_norm(x, normed=x, pre_weight=x[0]),
                 lambda: D.Fp8Rows(w.codes, w.scales[:, :2]), lambda: D.Fp8Rows(w.codes.T, w.scales), lambda: D.Fp8Rows(w.codes, w.scales.cpu())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: D.moe_fp8_linear(x, w, y, ws[:16]), lambda: D.moe_residual_norm(x), lambda: D.moe_residual_norm(x, normed=x, eps=0.0),
                 lambda: D.moe_residual_norm(x, y=x), lambda: D.moe_residual_norm(x, x, normed=x, y=x)):
        with pytest.raises(RuntimeError):
            call()
