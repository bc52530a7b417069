"""Attention over inputs at the edge of what a call may hold, and past it: what
only the device can see to be wrong."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import _native as N
from tests.test_gpu_attention import ints, make_cache, normal, run_cached, starts

pytestmark = pytest.mark.gpu
INVALID = 1


# (length, drafted): one tile, pieces that are joined, several pairs of tiles, and pairs that do not see the last pieces
@pytest.mark.parametrize("length,draft", [(300, 1), (2500, 2), (700, 300), (2500, 1500)])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("fp16", 128)])
def test_cached_bad_page_ids_undo_their_sequence_alone(cuda, length, draft, page, dtype, dim):
    """Wherever in the sequence the bad id stands, all of its queries give 0 and -inf, and the other sequences what
    they give without it."""
    lengths, drafts = [260, length, 1300, 90], [3, draft, 1, 5]
    cache = make_cache(lengths, 2, dim, page, dtype, 80)
    q = normal((sum(drafts), 4, dim), dtype, 81)
    seqs, cu = ints([0, 1, 2, 3]), starts(drafts)
    good, good_lse = run_cached(q, cache, 0, seqs, cu)
    assert N.check_status() == 0 and torch.isfinite(good.float()).all() and torch.isfinite(good_lse).all()
    mine = torch.zeros(sum(drafts), dtype=torch.bool, device="cuda")
    mine[drafts[0]:drafts[0] + draft] = True
    held = -(-length // page)
    for at in (0, held // 2, held - 1):
        page_id = int(cache.table[1, at])
        for bad in (-1, cache.pages.shape[1], 1 << 30):
            cache.table[1, at] = bad
            out, lse = run_cached(q, cache, 0, seqs, cu)
            assert N.check_status() == INVALID
            assert (out[mine] == 0).all() and (lse[mine] == -np.inf).all(), (at, bad)
            assert torch.equal(out[~mine], good[~mine]) and torch.equal(lse[~mine], good_lse[~mine])
        cache.table[1, at] = page_id
    out, lse = run_cached(q, cache, 0, seqs, cu)
    assert N.check_status() == 0 and torch.equal(out, good) and torch.equal(lse, good_lse)


@pytest.mark.parametrize("page", [16, 5])
def test_cached_bad_page_ids_under_a_mask(cuda, page):
    lengths, drafts = [40, 500], [7, 200]
    cache = make_cache(lengths, 1, 64, page, "bf16", 82)
    q = normal((sum(drafts), 2, 64), "bf16", 83)
    mask = torch.full((sum(drafts), 7), -1, dtype=torch.int32, device="cuda")
    good, _ = run_cached(q, cache, 1, ints([0, 1]), starts(drafts), mask)
    for at in (0, 499 // page):
        page_id = int(cache.table[1, at])
        cache.table[1, at] = -1
        out, lse = run_cached(q, cache, 1, ints([0, 1]), starts(drafts), mask)
        assert N.check_status() == INVALID
        assert (out[7:] == 0).all() and (lse[7:] == -np.inf).all() and torch.equal(out[:7], good[:7])
        cache.table[1, at] = page_id
