"""The serving example end to end: what its cache holds after prompts, forks,
drafted trees, ended sequences and compaction."""
import pytest
import torch

from examples import draft_decode as E
from nvfp4_block_scaled_gather_gb300 import attention as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def served(cuda):
    return E.run()


def test_cache_holds_the_kept_tokens(served):
    server, live, accepted = served
    c = server.cache
    assert min(accepted) >= 1 and len(accepted) == 3 * 3 + 2
    lengths = [len(live.get(i, ())) for i in range(E.MAX_SEQS)]
    assert c.length.tolist() == lengths
    pages = [-(-n // E.PAGE) for n in lengths]
    assert c.held.tolist() == pages
    used = [p for row, n in zip(c.table.tolist(), pages) for p in row[:n]]
    assert all(p == -1 for row, n in zip(c.table.tolist(), pages) for p in row[n:])
    # every page in use once; the first sequence's end left its pages to the ones behind, and later steps took more
    assert len(set(used)) == len(used) and min(used) == 0
    refs = c.refs.tolist()
    assert [p for p, r in enumerate(refs) if r] == sorted(used) and set(refs) <= {0, 1}


def test_first_block_rows_are_those_of_the_tokens(served):
    """The keys and values of the first block depend on the token alone. The product that makes them may be summed in
    another order for another number of rows: fp32 sums of 256 products of bf16 rounded to bf16, so an element is off
    by one unit in the last place (2^-7 of its size) where the two sums round apart, or by the sums' own error (256 *
    2^-24 of the sum of magnitudes, below 16 here) where the element nearly cancels."""
    server, live, _ = served
    c = server.cache
    for i, tokens in live.items():
        h = server.model.embed[torch.tensor(tokens, device="cuda")]
        x = (E.norm(h) @ server.model.qkv[0]).view(len(tokens), -1, E.DIM)
        table = c.table[i].tolist()
        rows = torch.tensor([table[t // E.PAGE] * E.PAGE + t % E.PAGE for t in range(len(tokens))], device="cuda")
        for plane, want in ((0, x[:, E.HEADS:E.HEADS + E.KV_HEADS]), (1, x[:, E.HEADS + E.KV_HEADS:])):
            got = c.pages[plane].flatten(0, 1)[rows].float()
            want = want.float()
            assert bool(((got - want).abs() <= want.abs() * 2 ** -7 + 256 * 2 ** -24 * 16).all())


@pytest.mark.parametrize("layer", range(E.LAYERS))
def test_cached_attention_equals_prompt_attention_over_the_kept_rows(served, layer):
    """A query at each live sequence's end, over the pages and over the same rows packed. Both round P to bf16 (2^-9
    relative a weight, at most, so 2^-9 of max |v| on the output) and the output to bf16 (2^-9 of it)."""
    server, live, _ = served
    c, seqs = server.cache, list(live)
    n = len(seqs)
    g = torch.Generator(device="cuda").manual_seed(layer)
    q = torch.randn((n, E.HEADS, E.DIM), device="cuda", generator=g).bfloat16()
    cached, packed = torch.empty_like(q), torch.empty_like(q)
    A.moe_attention_cached(q, c, layer, E.ints(seqs), E.starts([1] * n), cached, server.attn_ws)
    rows = [c.table[i].tolist()[t // E.PAGE] * E.PAGE + t % E.PAGE for i in seqs for t in range(len(live[i]))]
    rows = torch.tensor(rows, device="cuda")
    k, v = (c.pages[2 * layer + x].flatten(0, 1)[rows].contiguous() for x in (0, 1))
    A.moe_attention_prompt(q, k, v, E.starts([1] * n), E.starts([len(live[i]) for i in seqs]), packed)
    top = float(v.float().abs().max())
    assert float((cached.float() - packed.float()).abs().max()) <= 4 * 2 ** -9 * top
