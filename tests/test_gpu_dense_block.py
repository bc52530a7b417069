"""The dense operators as a decoder block uses them, between attention over the
paged cache and the routed experts; several streams at once; tensors past 2^31
elements."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import _native as N
from nvfp4_block_scaled_gather_gb300 import attention as A
from nvfp4_block_scaled_gather_gb300 import dense as D
from nvfp4_block_scaled_gather_gb300.synthetic import CONFIGS, make_weights
from tests.test_gpu_dense import gemm, norm_holds, normal, products_hold, quantize, whole_rows

pytestmark = pytest.mark.gpu

CFG = CONFIGS["tiny"]
HEADS, KV, DIM, VOCAB, PAGE = 8, 2, 64, 501, 16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Block:
    """One block of a decoder and its logits, all of it the library's but for the router."""

    def __init__(self):
        h = CFG.H
        self.qkv, self.back, self.logits = (quantize(normal((n, k), "bf16", i, k ** -0.5)) for i, (n, k) in enumerate(
            (((HEADS + 2 * KV) * DIM, h), (h, HEADS * DIM), (VOCAB, h))))
        self.router = normal((h, CFG.E), "bf16", 4, h ** -0.5)
        w = make_weights(CFG.E, h, CFG.I, seed=3, device="cuda")
        self.experts = N.MoeLayer(N.Weights(*(w[k] for k in ("w13_packed", "w13_sf_linear", "g_gate_up", "w2_packed",
                                                             "w2_sf_linear", "g_down"))), 64, CFG.k)
        self.norms = [1 + 0.1 * normal((n,), "fp32", 5 + i) for i, n in enumerate((h, DIM, h, h, h))]
        self.gate = torch.sigmoid(normal((h,), "fp32", 11)).bfloat16()
        self.cache = A.KVCache.empty(1, 64, PAGE, KV, DIM, 4, 16)
        self.pages_ws = A.pages_workspace(self.cache)
        self.attn_ws = A.cached_workspace(self.cache, 4, 64, HEADS)

    def __call__(self, x, seqs, counts, keep=None):
        """x [tokens, h], the tokens of each sequence next to each other; `keep` gets what the checks look at."""
        t, h = x.shape
        cu = ints([sum(counts[:i]) for i in range(len(counts) + 1)])
        rows, stream = D.Fp8Rows.empty(t, h), torch.empty_like(x)
        qkv = torch.empty((t, HEADS + 2 * KV, DIM), dtype=x.dtype, device="cuda")
        D.moe_residual_norm(x, quantized=rows, pre_weight=self.norms[0])
        D.moe_fp8_gemm(rows, self.qkv, qkv.view(t, -1))
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
        plain = qkv.clone() if keep is not None else None
        D.moe_residual_norm(qkv[:, :HEADS + KV], normed=qkv[:, :HEADS + KV], pre_weight=self.norms[1])
        A.moe_kv_extend(self.cache, ints(seqs), ints(counts), self.pages_ws)
        A.moe_kv_append(self.cache, 0, ints(seqs), cu, k, v)
        out = torch.empty((t, HEADS, DIM), dtype=x.dtype, device="cuda")
        A.moe_attention_cached(q, self.cache, 0, ints(seqs), cu, out, self.attn_ws)
        back = torch.empty_like(x)
        D.moe_fp8_linear(out.view(t, -1), self.back, back, D.linear_workspace(t, HEADS * DIM))
        normed = torch.empty_like(x)
        D.moe_residual_norm(x, back, y=stream, normed=normed, post_norm=True, post_weight=self.norms[2],
                            pre_weight=self.norms[3], gate=self.gate.view(1, h), residual_scale=0.5)
        weight, ids = torch.topk(torch.softmax((normed @ self.router).float(), -1), CFG.k)
        mixed = self.experts(normed, ids.int().contiguous(), weight.contiguous()).clone()
        last = D.Fp8Rows.empty(t, h)
        D.moe_residual_norm(stream, mixed, y=stream, quantized=last, pre_weight=self.norms[4])
        logits = torch.empty((t, VOCAB), device="cuda")
        D.moe_fp8_gemm(last, self.logits, logits)
        if keep is not None:
            keep.update(rows=rows, plain=plain, qkv=qkv, out=out, back=back, stream=stream, normed=normed, mixed=mixed, last=last,
                        logits=logits)
        return logits


@pytest.mark.parametrize("prompts", [[5, 11, 1], [40, 9, 15]])
def test_a_block_step_by_step(cuda, prompts):
    """Every step against 64 bits on the inputs that it had."""
    block, s = Block(), {}
    t = sum(prompts)
    x = normal((t, CFG.H), "bf16", 20, 2.0)
    block(x, [0, 1, 2], prompts, s)
    torch.cuda.synchronize()
    assert N.check_status() == 0
    norm_holds(x[:, None], None, dict(pre_weight=block.norms[0], eps=1e-6), "bf16", None, None, s["rows"])
    products_hold(s["plain"].view(t, -1), s["rows"], block.qkv, "bf16")
    norm_holds(s["plain"][:, :HEADS + KV], None, dict(pre_weight=block.norms[1], eps=1e-6), "bf16", None, s["qkv"][:, :HEADS + KV])
    assert torch.equal(s["plain"][:, HEADS + KV:], s["qkv"][:, HEADS + KV:])
    products_hold(s["back"], quantize(s["out"].view(t, -1)), block.back, "bf16")
    before = torch.empty_like(x)
    kw = dict(post_norm=True, post_weight=block.norms[2], pre_weight=block.norms[3], gate=block.gate.view(1, 1, -1), residual_scale=0.5,
              eps=1e-6)
    D.moe_residual_norm(x, s["back"], y=before, post_norm=True, post_weight=block.norms[2], gate=block.gate.view(1, -1), residual_scale=0.5)
    norm_holds(x[:, None], s["back"][:, None], kw, "bf16", before[:, None], s["normed"][:, None])
    norm_holds(before[:, None], s["mixed"][:, None], dict(pre_weight=block.norms[4], eps=1e-6), "bf16", s["stream"][:, None], None, s["last"])
    products_hold(s["logits"], s["last"], block.logits, "fp32")


def test_a_token_gives_the_same_logits_alone_and_in_a_batch(cuda):
    """No step of the block looks at the other sequences: decoding one after the other gives the bits of decoding them
    together."""
    prompts = [7, 20, 3]
    x, y = normal((30, CFG.H), "bf16", 30, 2.0), normal((3, CFG.H), "bf16", 31, 2.0)
    together, apart = Block(), Block()
    together(x, [0, 1, 2], prompts)
    want = together(y, [0, 1, 2], [1, 1, 1])
    at = 0
    for i, n in enumerate(prompts):
        apart(x[at:at + n], [i], [n])
        at += n
        # (the router's product is torch's: its sums may differ with the number of rows, by far less than makes a choice)
        assert torch.equal(apart(y[i:i + 1], [i], [1]), want[i:i + 1])


def test_products_on_several_streams_at_once(cuda):
    """Pairs, clusters and single CTAs side by side on one GPU, each with buffers of its own."""
    shapes = [(300, 1000, 2064), (1, 5000, 4096), (64, 384, 8192), (700, 2000, 1024), (20, 20000, 1024), (130, 100, 512)]
    sets = []
    for t, n, k in shapes:
        x, w = whole_rows(t, k, t, 2), whole_rows(n, k, n, 2)
        sets.append((x, w, torch.zeros((t, n), device="cuda"), (x.dequantized().double() @ w.dequantized().double().T).float(),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, y, _, s in sets:
            with torch.cuda.stream(s):
                D.moe_fp8_gemm(x, w, y)
    torch.cuda.synchronize()
    assert N.check_status() == 0
    for _, _, y, want, _ in sets:
        assert torch.equal(y, want)


def test_results_past_32_bits(cuda):
    """More than 2^31 results: their offsets need 64 bits."""
    t, n, k = 70001, 32000, 16
    x, w = whole_rows(t, k, 1), whole_rows(n, k, 2)
    y = torch.full((t, n), 7.0, dtype=torch.float16, device="cuda")
    assert y.numel() > 2 ** 31
    D.moe_fp8_gemm(x, w, y)
    xs, ws = x.dequantized(), w.dequantized()
    for a in (0, 33000, 67107, t - 300):  # (67107 * 32000 is the last row below 2^31)
        assert torch.equal(y[a:a + 300].float(), xs[a:a + 300] @ ws.T)
    assert N.check_status() == 0


def test_rows_past_32_bits(cuda):
    """More than 2^31 bytes of codes, as tokens and as rows of w, and their quantization."""
    rows, k = 135000, 16384
    big = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    picks = [0, 1, 131071, 131072, 131073, rows - 1]
    some = normal((len(picks), k), "bf16", 1)
    big[torch.tensor(picks, device="cuda")] = some
    q = D.Fp8Rows.empty(rows, k)
    D.moe_fp8_quantize_rows(big, q)
    del big
    small = quantize(some)
    at = torch.tensor(picks, device="cuda")
    assert torch.equal(q.codes.view(torch.uint8)[at], small.codes.view(torch.uint8)) and torch.equal(q.scales[at], small.scales)
    other = quantize(normal((130, k), "bf16", 2, k ** -0.5))
    want = gemm(small, other)
    y = torch.empty((rows, 130), device="cuda")
    D.moe_fp8_gemm(q, other, y)
    assert torch.equal(y[at], want) and int((y != 0).any(1).sum()) == len(picks)
    y = torch.empty((130, rows), device="cuda")
    D.moe_fp8_gemm(other, q, y)
    assert torch.equal(y[:, at], gemm(other, small)) and N.check_status() == 0


def test_norms_past_32_bits(cuda):
    t, d = 530000, 4096
    x = torch.zeros((t, d), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 524287, 524288, 524289, t - 1], device="cuda")
    some = normal((5, d), "bf16", 1)
    x[at] = some
    want = torch.empty_like(some)
    D.moe_residual_norm(some, normed=want)
    D.moe_residual_norm(x, normed=x)
    assert torch.equal(x[at], want)
    x[at] = 0
    assert not x.any() and N.check_status() == 0
    heads = x.view(-1, 64)[:, None]  # rows of 64: 33 million
    heads[-3:] = normal((3, 1, 64), "bf16", 2)
    one = torch.empty((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    D.moe_residual_norm(heads[-3:], normed=one)
    D.moe_residual_norm(heads, normed=heads)
    assert torch.equal(heads[-3:], one) and not heads[:-3].any()


def test_calls_captured_together_share_a_workspace_in_stream_order(cuda):
    """Two graphs over one workspace, replayed one after the other: the second's rows are its own."""
    w = quantize(normal((640, 2048), "bf16", 1, 0.02))
    ws = D.linear_workspace(200, 2048)
    graphs, sets = [], []
    for seed in (3, 4):
        x, y = normal((200, 2048), "bf16", seed), torch.zeros((200, 640), device="cuda")
        D.moe_fp8_linear(x, w, y, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            D.moe_fp8_linear(x, w, y, ws)
        graphs.append(g)
        sets.append((x, y))
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for x, y in sets:
        assert torch.equal(y, gemm(quantize(x), w))
    assert N.check_status() == 0


def test_a_large_step_of_everything_beside_attention_is_deterministic(cuda):
    x, b = normal((900, 4096), "bf16", 1), normal((900, 4096), "bf16", 2)
    w = quantize(normal((3000, 4096), "bf16", 3, 4096 ** -0.5))
    first = None
    for _ in range(4):
        rows, y = D.Fp8Rows.empty(900, 4096), torch.empty_like(x)
        out = torch.empty((900, 3000), dtype=torch.bfloat16, device="cuda")
        D.moe_residual_norm(x, b, y=y, quantized=rows, post_norm=True)
        D.moe_fp8_gemm(rows, w, out)
        got = (y, rows.codes.view(torch.uint8), rows.scales, out)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    assert np.isfinite(out.float().sum().item())
