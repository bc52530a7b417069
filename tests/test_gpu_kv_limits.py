"""Upkeep of the paged cache at its limits: state that only the device can see
to be wrong, requests that no pool can serve, long lists."""
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import _native as N
from nvfp4_block_scaled_gather_gb300 import attention as A

pytestmark = pytest.mark.gpu
INVALID, OUT_OF_PAGES = 1, 6
LEAST = -2 ** 31


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("length,held", [(-1, 2), (-100, 2), (LEAST, 2), (LEAST, LEAST), (20, -1), (-3, -3)])
def test_counts_below_zero_are_reported_and_not_followed(cuda, length, held):
    """A sequence whose counts are of no sequence is left alone by all upkeep, and so is what lies around its rows."""
    cache = A.KVCache.empty(1, 12, 16, 1, 8, 4, 3)
    ws = A.pages_workspace(cache)
    A.moe_kv_extend(cache, ints([0, 1, 2, 3]), ints([40, 20, 33, 5]), ws)
    cache.pages.copy_(torch.randn_like(cache.pages))
    assert N.check_status() == 0
    cache.length[1], cache.held[1] = length, held
    state = (cache.table, cache.length, cache.held, cache.refs, cache.pages)
    before = [t.clone() for t in state]
    one, rows = ints([1]), torch.randn((1, 1, 8), device="cuda").bfloat16()
    for name, call in (("truncate", lambda: A.moe_kv_truncate(cache, one, ints([0]))),
                       ("cut", lambda: A.moe_kv_truncate(cache, one, ints([7]))),
                       ("keep", lambda: A.moe_kv_keep(cache, one, ints([1]), ints([[0]]), ints([1]), ws)),
                       ("keep none", lambda: A.moe_kv_keep(cache, one, ints([2]), ints([[0]]), ints([0]), ws)),
                       ("append", lambda: A.moe_kv_append(cache, 0, one, ints([0, 1]), rows, rows)),
                       ("extend", lambda: A.moe_kv_extend(cache, one, ints([1]), ws))):
        if name.startswith(("append", "keep")) and length >= 0:
            continue  # these go by the length and the table alone
        call()
        assert N.check_status() == INVALID, name
        assert all(torch.equal(a, b) for a, b in zip(state, before)), name


def wide_cache(n_pages, max_seqs, max_pages):
    """A fresh cache of one-token pages whose table is not filled (nothing of it is read where a sequence is empty)."""
    zeros = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return A.KVCache(torch.zeros((2, n_pages, 1, 1, 8), dtype=torch.bfloat16, device="cuda"),
                     torch.empty((max_seqs, max_pages), dtype=torch.int32, device="cuda"), zeros(max_seqs), zeros(max_seqs),
                     zeros(n_pages))


@pytest.mark.parametrize("n,each", [(2, 1 << 30), (1500, 1 << 21), (1024, (1 << 21) + 1)])
def test_wants_that_pass_32_bits_are_out_of_pages(cuda, n, each):
    """Together 2^31 and more pages, in one pass of the plan's threads and in two: all or nothing."""
    cache = wide_cache(5, n, each)
    ws = A.pages_workspace(cache)
    assert N.check_status() == 0
    A.moe_kv_extend(cache, ints(list(range(n))), ints([each] * n), ws)
    assert N.check_status() == OUT_OF_PAGES
    assert not cache.length.any() and not cache.held.any() and not cache.refs.any()
    A.moe_kv_extend(cache, ints([0, 1]), ints([2, 3]), ws)
    assert N.check_status() == 0
    assert cache.length[:3].tolist()[:2] == [2, 3] and cache.refs.tolist() == [1] * 5
    assert cache.table[0, :2].tolist() == [0, 1] and cache.table[1, :3].tolist() == [2, 3, 4]


def test_copies_of_more_pages_than_a_call_has_sequences(cuda):
    n = 5000
    cache = A.KVCache.empty(1, 2 * n, 2, 1, 8, 1, 1)
    cache.pages.copy_(torch.randn_like(cache.pages))
    want = cache.pages[:, :n].flip(1).clone()
    A.moe_kv_copy_pages(cache, torch.arange(n, dtype=torch.int32, device="cuda"),
                        torch.arange(2 * n - 1, n - 1, -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(cache.pages[:, n:], want) and N.check_status() == 0
