"""Attention over inputs at the edge of what a call may hold, and past it: what
only the device can see to be wrong."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import _native as N
from nvfp4_block_scaled_gather_gb300 import attention as A
from oracle import attention as OA
from tests.test_gpu_attention import f64, hold, ints, make_cache, normal, run_cached, starts

pytestmark = pytest.mark.gpu
INVALID = 1
LEAST, MOST = -2 ** 31, 2 ** 31 - 1


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


def guarded(q, k, v, cu_q, cu_k):
    """Prompt attention into the middle of larger tensors: results, after the rows around them were found untouched."""
    n, heads, dim = q.shape
    out = torch.full((n + 64, heads, dim), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((n + 64, heads), 7.0, dtype=torch.float32, device="cuda")
    A.moe_attention_prompt(q, k, v, ints(cu_q), ints(cu_k), out[32:32 + n], lse=lse[32:32 + n])
    torch.cuda.synchronize()
    assert N.check_status() == 0
    for x in (out, lse):
        assert (x[:32] == 7).all() and (x[32 + n:] == 7).all()
    return out[32:32 + n], lse[32:32 + n]


@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_offsets_are_cut_to_the_tensors(cuda, dim):
    """(rows, keys) of each sequence, from offsets that lie outside the tensors, run backwards or differ by more than
    32 bits hold. Rows of no sequence are left alone."""
    q, k, v = normal((40, 2, dim), "bf16", 33), normal((40, 2, dim), "bf16", 34), normal((40, 2, dim), "bf16", 35)
    none = (0, 0)
    for cu_q, cu_k, want in (
            ([-5, 10, 1000], [0, 20, 30], [((0, 10), (0, 20)), ((10, 40), (20, 30))]),
            ([0, 20, 1000], [0, 500, 30], [((0, 20), (0, 40)), ((20, 40), none)]),
            ([5, LEAST], [0, 40], []),
            ([MOST, LEAST], [0, 40], []),
            ([MOST, 12], [0, 40], []),
            ([30, 4, 4], [0, 10, 40], []),
            ([0, 40], [7, LEAST], [((0, 40), none)]),
            ([0, 40], [MOST, LEAST], [((0, 40), none)]),
            ([0, 15, 40], [MOST, 7, LEAST], [((0, 15), none), ((15, 40), none)]),
            ([LEAST, MOST], [LEAST, MOST], [((0, 40), (0, 40))])):
        out, lse = guarded(q, k, v, cu_q, cu_k)
        mine = torch.zeros(40, dtype=torch.bool, device="cuda")
        for (a, b), (c, d) in want:
            mine[a:b] = True
            hold(out[a:b], lse[a:b], q[a:b], k[c:d], v[c:d], OA.chain(b - a, d - c), dim ** -0.5, "bf16")
        assert (out[~mine] == 7).all() and (lse[~mine] == 7).all()


def test_cached_offsets_are_cut_to_the_tensors(cuda):
    cache = make_cache([2000, 300], 2, 64, 16, "bf16", 36)
    q = normal((30, 4, 64), "bf16", 37)
    whole, whole_lse = run_cached(q, cache, 0, ints([0]), ints([0, 30]))
    for cu, rows in (([5, LEAST], 0), ([MOST, LEAST], 0), ([LEAST, MOST], 30), ([-1, 31], 30)):
        out, lse = run_cached(q, cache, 0, ints([0]), ints(cu))
        assert torch.equal(out[:rows], whole[:rows]) and torch.equal(lse[:rows], whole_lse[:rows])
        assert (out[rows:] == 7).all() and (lse[rows:] == 7).all() and N.check_status() == 0


@pytest.mark.parametrize("cu,status", [([3, LEAST], 0), ([MOST, LEAST], 0), ([MOST, 2], 0), ([6, 2], 0), ([LEAST, 6], INVALID),
                                       ([LEAST, MOST], INVALID)])
def test_tree_mask_offsets_that_hold_no_tokens(cuda, cu, status):
    parents = torch.full((64 + 6 + 64,), -1, dtype=torch.int32, device="cuda")[64:70]
    mask = torch.full((64 + 6 + 64, 1), 77, dtype=torch.int32, device="cuda")
    A.moe_tree_mask(parents, ints(cu), mask[64:70])
    torch.cuda.synchronize()
    assert N.check_status() == status and (mask == 77).all()


def test_offsets_that_give_every_row_to_thousands_of_sequences(cuda):
    """2^19 pairs of one-token tiles for each of 10000 sequences: more items than 32 bits count. Nothing is done."""
    total, n = 1 << 20, 20001
    x = torch.zeros((total, 128, 8), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 7.0)
    cu = torch.zeros(n, dtype=torch.int32, device="cuda")
    cu[1::2] = total
    A.moe_attention_prompt(x, x[:64, :1], x[:64, :1], cu, torch.zeros_like(cu), out)
    torch.cuda.synchronize()
    assert N.check_status() == INVALID and (out == 7).all()
    q, few = normal((300, 2, 64), "bf16", 39), [0] * 300 + [200, 100, 300]  # 100 queries twice, 303 offsets
    less = torch.full_like(q, 7.0)
    A.moe_attention_prompt(q, q, q, ints(few), ints(few), less)
    assert N.check_status() == INVALID and (less == 7).all()
    cache = make_cache([2000], 1, 8, 16, "bf16", 38)
    ws = A.cached_workspace(cache, n - 1, total, 128).zero_()
    A.moe_attention_cached(x, cache, 0, torch.zeros(n - 1, dtype=torch.int32, device="cuda"), cu, out, ws)
    torch.cuda.synchronize()
    assert N.check_status() == INVALID and (out == 7).all()


def test_other_devices_are_refused(cuda, monkeypatch):
    """Tensors of a device that is not the current one, and streams of another: nothing is launched."""
    q, cu = normal((3, 4, 64), "bf16", 84), ints([0, 3])
    kv, out = normal((3, 2, 64), "bf16", 85), torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    cache = A.KVCache.empty(1, 4, 16, 2, 64, 2, 4)
    ws, seqs, three = A.pages_workspace(cache), ints([0]), ints([3])
    attn_ws, mask, places = A.cached_workspace(cache, 1, 3, 4), ints([[0]] * 3), ints([[0]])

    class Elsewhere:
        cuda_stream, device = 0, torch.device("cuda", 1)

    def calls(**stream):
        return (lambda: A.moe_attention_prompt(q, kv, kv, cu, cu, out, **stream),
                lambda: A.moe_attention_cached(q, cache, 0, seqs, cu, out, attn_ws, **stream),
                lambda: A.moe_kv_extend(cache, seqs, three, ws, **stream),
                lambda: A.moe_kv_append(cache, 0, seqs, cu, kv, kv, **stream),
                lambda: A.moe_kv_fork(cache, seqs, ints([1]), **stream),
                lambda: A.moe_kv_truncate(cache, seqs, three, **stream),
                lambda: A.moe_kv_keep(cache, seqs, three, places, seqs, ws, **stream),
                lambda: A.moe_kv_copy_pages(cache, seqs, three, **stream),
                lambda: A.moe_kv_compact(cache, ws, **stream),
                lambda: A.moe_tree_mask(ints([-1, 0, 1]), cu, mask, **stream))

    for call in calls(stream=Elsewhere()):
        with pytest.raises(ValueError, match="device"):
            call()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in calls():
        with pytest.raises(ValueError, match="device"):
            call()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert (out == 7).all() and not cache.refs.any() and not cache.length.any() and N.check_status() == 0


@pytest.mark.parametrize("call", ["prompt", "cached"])
@pytest.mark.parametrize("n", [2000, 40000])
def test_small_weights_of_fp16_count(cuda, call, n):
    """One key of weight 1 whose value is 0, and n - 1 of weight 2^-26 with values of 1. In fp16 half of the least
    number above 0 is 2^-25, so weights that are held as they are would leave nothing of them. Each is a power of two
    and has no rounding error of its own; the scores' is 2^-20 (a product of 64 terms below 2^5 in fp32: 72 * 2^-22 * 2^5
    is 2^-10.8 of a weight), the output's 2^-11 and, below fp16's normal numbers, 2^-25."""
    dim = 64
    q, k, v = (torch.zeros((m, 1, dim)) for m in (1, n, n))
    q[:] = 1.0
    k[n // 3, 0, 0] = 26.0            # in powers of two, by the scale
    v[:] = 1.0
    v[n // 3] = 0.0
    q, k, v = (x.half().cuda() for x in (q, k, v))
    scale = float(np.log(2.0))
    if call == "prompt":
        out, lse = torch.empty_like(q), torch.empty((1, 1), device="cuda")
        A.moe_attention_prompt(q, k, v, ints([0, 1]), ints([0, n]), out, lse=lse, scale=scale)
    else:
        cache = A.KVCache.empty(1, -(-n // 64), 64, 1, dim, 1, -(-n // 64), dtype=torch.float16)
        A.moe_kv_extend(cache, ints([0]), ints([n]), A.pages_workspace(cache))
        A.moe_kv_append(cache, 0, ints([0]), ints([0, n]), k, v)
        out, lse = run_cached(q, cache, 0, ints([0]), ints([0, 1]), scale=scale)
    rest = (n - 1) * 2.0 ** -26
    want = rest / (1.0 + rest)
    assert np.abs(f64(out) - want).max() <= want * (2.0 ** -10.8 + 2.0 ** -11) + 2.0 ** -25
    assert abs(float(lse) - (26.0 * np.log(2.0) + np.log1p(rest))) <= 2.0 ** -10.8 + 2.0 ** -20 * 20


@pytest.mark.parametrize("context", [0, 3000])
def test_values_that_are_not_finite_in_a_mask_of_thousands_of_tokens(cuda, context):
    """They reach the rows that see them, whichever those are, and the call ends in time."""
    n, dim, page = 16000, 128, 64
    cache = make_cache([context + n], 1, dim, page, "bf16", 40, layers=1)
    g = torch.Generator(device="cuda").manual_seed(41)
    mask = torch.randint(LEAST, MOST, (n, n // 32), dtype=torch.int32, device="cuda", generator=g)
    places = {5: float("inf"), n // 2: float("nan"), n - 2: -float("inf"), n - 1: float("inf")}
    columns = {5: 3, n // 2: 100, n - 2: 64, n - 1: 64}
    for j, value in places.items():
        at = context + j
        cache.pages[1, int(cache.table[0, at // page]), at % page, 0, columns[j]] = value
    out, lse = run_cached(normal((n, 1, dim), "bf16", 42), cache, 0, ints([0]), ints([0, n]), mask)
    assert N.check_status() == 0 and torch.isfinite(lse).all()
    sees = {j: (mask[:, j // 32] >> (j % 32) & 1) != 0 for j in places}
    want = torch.zeros((n, dim), device="cuda")
    for j, value in places.items():
        want[:, columns[j]] += torch.where(sees[j], value, 0.0)
    got = torch.where(torch.isfinite(out[:, 0].float()), 0.0, out[:, 0].float())
    assert torch.equal(torch.nan_to_num(got, 1.0, 2.0, 3.0), torch.nan_to_num(want, 1.0, 2.0, 3.0))


def test_masks_without_words_are_refused(cuda):
    """They have no address, and without one a call is a chain, whose tokens see those before them."""
    cache = make_cache([20], 1, 64, 16, "bf16", 43)
    q = normal((4, 2, 64), "bf16", 44)
    out, ws = torch.empty_like(q), A.cached_workspace(cache, 1, 4, 2)
    with pytest.raises(ValueError, match="word"):
        A.moe_attention_cached(q, cache, 0, ints([0]), ints([0, 4]), out, ws, mask=torch.empty((4, 0), dtype=torch.int32, device="cuda"))
    A.moe_attention_cached(q[:0], cache, 0, ints([0]), ints([0, 0]), out[:0], ws,
                           mask=torch.empty((0, 0), dtype=torch.int32, device="cuda"))
