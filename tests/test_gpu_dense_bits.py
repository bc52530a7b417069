"""The bits of the dense products, where comparing values does not see them: zeros' signs, all 24 bits of a sum; and the kernel
that quantizes up to 32 tokens on the way."""
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import _native as N
from nvfp4_block_scaled_gather_gb300 import dense as D
from tests.test_gpu_dense import gemm, normal, quantize

pytestmark = pytest.mark.gpu

INTS = {"bf16": torch.int16, "fp16": torch.int16, "fp32": torch.int32}


def rows_of(rows, k, code, scale):
    return D.Fp8Rows(torch.full((rows, k), code, dtype=torch.uint8, device="cuda"),
                     torch.full((rows, 4 * -(-k // 512)), scale, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n,k", [(640, 4096), (200, 9216), (1100, 528), (20000, 1024)])
def test_zeros_have_one_sign_whatever_the_batch(cuda, n, k, dtype):
    """Products that are all -0, and negative ones below fp32's smallest: the same bits in clusters, pairs and single CTAs."""
    for x, w in ((rows_of(600, k, 0x80, 127), rows_of(n, k, 0x38, 127)), (rows_of(600, k, 0x01, 0), rows_of(n, k, 0x81, 0))):
        want = gemm(x, w, dtype).view(INTS[dtype])
        for t in (1, 8, 16, 30, 40, 64, 128, 300):
            assert torch.equal(gemm(x.rows(t), w, dtype).view(INTS[dtype]), want[:t]), t


def quantized_on_the_way(x, w, out="bf16"):
    """moe_fp8_linear's result, and whether it left its workspace as it was: calls that quantize on the way do."""
    t, k = x.shape
    y, ws = torch.empty((t, w.n), dtype=getattr(torch, {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}[out]), device="cuda"), None
    ws = torch.full((D.load().moe_fp8_linear_workspace_size(t, k),), 255, dtype=torch.uint8, device="cuda")
    D.moe_fp8_linear(x, w, y, ws)
    torch.cuda.synchronize()
    assert N.check_status() == 0
    return y, bool((ws == 255).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("t,n,k", [(32, 4096, 4096), (17, 2570, 1040), (25, 6144, 2048), (18, 4097, 512 * 7 + 16), (31, 2600, 4080)])
def test_up_to_32_tokens_quantized_on_the_way(cuda, t, n, k, dtype):
    """Tiles of 32 tokens, where those of 16 would be more clusters than run at one time."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert t > 16 and -(-n // 128) * 2 * 8 > 2 * sms  # (what the rule gives the tiles of 16 tokens)
    x, w = normal((t, k), dtype, t), quantize(normal((n, k), "bf16", n, k ** -0.5))
    x[t // 2, k // 3] = float("inf")
    x[t - 1, :128] = 0.0
    y, on_the_way = quantized_on_the_way(x, w, dtype)
    assert on_the_way
    want = gemm(quantize(x), w, dtype)
    whole = torch.arange(t, device="cuda") != t // 2
    assert torch.equal(y[whole].view(torch.int16), want[whole].view(torch.int16))
    assert torch.isnan(y[t // 2]).all() and torch.isnan(want[t // 2]).all() and torch.isfinite(y[whole]).all()


def odd_rows(rows, k, seed, signs=False):
    """Odd whole numbers of 9 to 15 under scales of 1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = 9.0 + 2 * torch.randint(0, 4, (rows, k), device="cuda", generator=g)
    if signs:
        v *= torch.randint(0, 2, (rows, k), device="cuda", generator=g) * 2 - 1
    return D.Fp8Rows(v.to(torch.float8_e4m3fn), torch.full((rows, 4 * -(-k // 512)), 127, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("t,n", [(1, 300), (16, 20000), (30, 2570), (40, 300), (300, 1000)])
def test_sums_keep_all_24_bits(cuda, t, n, signs):
    """Whole numbers, of which a block of 128 counts 512 times, another 32 and one 4 times, in another order in each row: sums
    of up to 128 * 225 * (512 + 32 + 4 + 1) + 16 * 225 < 2^24, most of them above 2^23, whose last bit is a single product's.
    Exact in fp32 whatever the order."""
    k = 656
    x, w = odd_rows(t, k, t, signs), odd_rows(n, k, n)
    g = torch.Generator(device="cuda").manual_seed(t + n)
    order = torch.stack([torch.randperm(5, device="cuda", generator=g) for _ in range(t)])
    x.scales[:, :5] = 127 + torch.tensor([0, 2, 5, 9, 0], dtype=torch.uint8, device="cuda")[order]
    want = x.dequantized().double() @ w.dequantized().double().T
    most = float((x.dequantized().double().abs() @ w.dequantized().double().T).max())
    assert 2 ** 23 < most < 2 ** 24
    assert torch.equal(gemm(x, w), want.float()) and torch.equal(want.float().double(), want)


@pytest.mark.parametrize("t,n,k", [(31, 12800, 1024), (32, 19000, 640), (17, 10000, 1024)])
def test_tokens_of_tiles_that_no_cluster_shares_are_quantized_once(cuda, t, n, k):
    """Else every CTA would do it again for all of K."""
    x, w = normal((t, k), "bf16", t), quantize(normal((n, k), "bf16", n, k ** -0.5))
    y, on_the_way = quantized_on_the_way(x, w)
    assert not on_the_way and torch.equal(y, gemm(quantize(x), w, "bf16"))


@pytest.mark.parametrize("n", [4608, 4609, 4864, 9472, 9473, 9728])
@pytest.mark.parametrize("t", [1, 30, 64])
def test_tiles_about_as_many_as_clusters_at_one_time(cuda, t, n):
    """A few more or less than the clusters of eight and four CTAs that run at one time: the bits of a row do not tell."""
    x, w = quantize(normal((t, 4096), "bf16", t)), quantize(normal((n, 4096), "bf16", n, 4096 ** -0.5))
    got = gemm(x, w)
    for a, b in ((0, 128), (n - 200, n)):
        some = D.Fp8Rows(w.codes[a:b], w.scales[a:b])
        assert torch.equal(got[:, a:b].contiguous().view(torch.int32), gemm(x, some).view(torch.int32))
    assert torch.equal(gemm(x.rows(1), w).view(torch.int32), got[:1].view(torch.int32))


@pytest.mark.parametrize("t,n,k,want", [(1, 512, 16384, False), (16, 512, 65536, False), (64, 512, 16384, False), (9, 64, 1 << 18, False),
                                        (16, 512, 8192, True), (1, 4096, 11008, True), (1, 8192, 16384, True), (300, 100, 11008, False), (500, 100, 11008, True)])
def test_a_long_k_is_quantized_on_the_way_where_reading_w_takes_as_long(cuda, t, n, k, want):
    """Up to 1024 + (n + 4 t) k / 32768 values of K a CTA, of eight pieces of K (four of which 64 tiles of w share): 300 x 100 x
    11,008 has 1536 and may have 1460, 500 x 100 may have 1729, 8192 x 16,384 has 4096 and may have 5122."""
    x, w = normal((t, k), "bf16", t), quantize(normal((n, k), "bf16", n, k ** -0.5))
    y, on_the_way = quantized_on_the_way(x, w)
    assert on_the_way == want
    assert torch.equal(y.view(torch.int16), gemm(quantize(x), w, "bf16").view(torch.int16))
