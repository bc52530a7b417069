"""Attention over whole prompts and over a paged cache, through the public
binding, against the definition in float64 with bounds derived from the
rounding of the weights and the output (oracle.attention.tolerance), at the
sizes and masks where it can go wrong."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import _native as N
from nvfp4_block_scaled_gather_gb300 import attention as A
from oracle import attention as OA

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def starts(lengths, first=0):
    return ints(np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int64).tolist())


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DTYPES[dtype]).cuda()


def f64(t):
    return t.double().cpu().numpy()


def hold(got_out, got_lse, q, k, v, seen, scale, dtype):
    """One sequence's results against the definition."""
    if not len(q):
        return
    out, lse, spread, product = OA.attention(f64(q), f64(k), f64(v), seen, scale)
    finite_v = f64(v)
    finite_v = np.abs(finite_v[np.isfinite(finite_v)])
    tol, tol_lse = OA.tolerance(out, lse, spread, product, q.shape[2], max(seen.shape[1], 1), dtype,
                                finite_v.max() if finite_v.size else 0.0)
    got, ge = f64(got_out), got_lse.double().cpu().numpy()
    fine = np.isfinite(out)
    assert np.array_equal(fine, np.isfinite(got))
    assert np.array_equal(np.isnan(out), np.isnan(got)) and np.array_equal(out[np.isinf(out)], got[np.isinf(out)])
    err = np.abs(got[fine] - out[fine])
    assert (err <= tol[fine]).all(), float((err / tol[fine]).max())
    there = np.isfinite(lse)
    assert np.array_equal(there, np.isfinite(ge)) and np.array_equal(lse[np.isinf(lse)], ge[np.isinf(lse)])
    assert (np.abs(ge[there] - lse[there]) <= tol_lse[there]).all()


def run_prompt(q, k, v, cu_q, cu_k, scale=None, stream=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda")
    A.moe_attention_prompt(q, k, v, cu_q, cu_k, out, lse=lse, scale=scale, stream=stream)
    return out, lse


def check_prompt(nq, nk, heads, kv, dim, dtype, seed=0, scale=None, spread=1.0):
    q, k, v = (normal((sum(m), h, dim), dtype, seed + i, s) for i, (m, h, s) in
               enumerate([(nq, heads, spread), (nk, kv, 1.0), (nk, kv, 1.0)]))
    out, lse = run_prompt(q, k, v, starts(nq), starts(nk), scale)
    torch.cuda.synchronize()
    assert N.check_status() == 0
    a = b = 0
    for n, m in zip(nq, nk):
        hold(out[a:a + n], lse[a:a + n], q[a:a + n], k[b:b + m], v[b:b + m], OA.chain(n, m),
             dim ** -0.5 if scale is None else scale, dtype)
        a, b = a + n, b + m


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 64), (4, 4, 128), (8, 1, 128), (6, 2, 80), (7, 1, 8), (20, 1, 64),
                                          (2, 2, 120), (128, 1, 64), (5, 1, 128)])
def test_prompt_head_layouts(cuda, dtype, heads, kv, dim):
    check_prompt([1, 37, 130], [1, 37, 130], heads, kv, dim, dtype)


@pytest.mark.parametrize("nq,nk", [
    ([0], [0]), ([0, 1, 0, 2, 0], [0, 1, 5, 2, 0]), ([127], [127]), ([128], [128]), ([129], [129]), ([255, 1], [255, 1]),
    ([256], [256]), ([257], [257]), ([385], [385]), ([1], [1000]), ([3], [129]), ([130], [259]), ([33, 64], [200, 64]),
    ([10], [4]), ([300], [20]), ([5, 9], [0, 3]), ([140, 140], [12, 400]),
])
def test_prompt_lengths(cuda, nq, nk):
    """Ends inside a tile, more keys than queries, fewer (queries that see no key), none at all."""
    check_prompt(nq, nk, 4, 2, 64, "bf16", seed=3)
    check_prompt(nq, nk, 2, 2, 128, "fp16", seed=4)


def test_prompt_many_sequences(cuda):
    rng = np.random.RandomState(0)
    nq = rng.randint(0, 9, 700).tolist()
    check_prompt(nq, [n + int(x) for n, x in zip(nq, rng.randint(0, 3, 700))], 2, 1, 64, "bf16", seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_prompt_sharp_and_large_scores(cuda, dtype):
    """Scores of hundreds: the running maximum moves by much, weights underflow."""
    check_prompt([300], [300], 2, 1, 128, dtype, seed=6, spread=20.0)
    check_prompt([200], [260], 2, 1, 64, dtype, seed=7, scale=3.0)
    check_prompt([90], [90], 2, 1, 64, dtype, seed=8, scale=1e-6)


def test_prompt_rising_scores(cuda):
    """Every block of keys has a larger maximum than the last: the accumulators are rescaled each time."""
    n, dim = 700, 64
    q, k, v = torch.ones((n, 1, dim)), torch.ones((n, 1, dim)), normal((n, 1, dim), "bf16", 9)
    k *= (torch.arange(n) // 16).float()[:, None, None] * 0.25
    q, k = q.bfloat16().cuda(), k.bfloat16().cuda()
    out, lse = run_prompt(q, k, v, starts([n]), starts([n]), 1.0)
    hold(out, lse, q, k, v, OA.chain(n, n), 1.0, "bf16")


def test_prompt_strided_inputs_and_packing_offsets(cuda):
    """q, k and v as slices of one projection's output; sequences that begin past row 0; heads in another order;
    rows outside the sequences left alone."""
    nq, lead, dim = [70, 200], 5, 64
    total = lead + sum(nq) + 3
    fused = normal((total, 8, dim), "bf16", 11)
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    cu = starts(nq, lead)
    out, lse = run_prompt(q, k, v, cu, cu)
    buffer = torch.full((4, total, dim), 7.0, dtype=torch.bfloat16, device="cuda")  # [heads, tokens, dim]
    other = buffer.transpose(0, 1)
    A.moe_attention_prompt(q, k, v, cu, cu, other)
    assert torch.equal(other, out)
    assert (out[:lead] == 7).all() and (out[-3:] == 7).all() and (lse[:lead] == 7).all() and (lse[-3:] == 7).all()
    a = lead
    for n in nq:
        hold(out[a:a + n], lse[a:a + n], q[a:a + n], k[a:a + n], v[a:a + n], OA.chain(n, n), dim ** -0.5, "bf16")
        a += n


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "fp16"), (80, "bf16")])
def test_prompt_poison_in_unseen_places(cuda, poison, dim, dtype):
    """Values that a query does not see do not reach it: later tokens of its own sequence, other sequences, rows
    around them; and what it does see does."""
    nq, lead = [150, 200], 3
    total = lead + sum(nq) + 40
    q, k, v = (normal((total, 2, dim), dtype, 20 + i) for i in range(3))
    v[:lead] = poison
    k[:lead] = poison
    v[lead + sum(nq):] = poison
    k[lead + sum(nq):] = poison
    v[lead + 77, 0, 3] = poison
    v[lead + 149] = poison
    k[lead + 150 + 90, 1] = poison if poison != float("-inf") else float("nan")
    v[lead + 150 + 130, 1, dim - 1] = poison
    v[lead + 150 + 131, 1, dim - 1] = -poison
    cu = starts(nq, lead)
    out, lse = run_prompt(q, k, v, cu, cu)
    a = lead
    for n in nq:
        seen = OA.chain(n, n)
        # the score of a poisoned key can come out as +-inf or NaN: hold what is before it, and that what is after is not finite
        clean = n if a == lead else 90
        hold(out[a:a + clean], lse[a:a + clean], q[a:a + clean], k[a:a + n], v[a:a + n], seen[:clean], dim ** -0.5, dtype)
        a += n
    late = out[lead + 150 + 90:lead + sum(nq), 1]
    assert not torch.isfinite(late.float().sum(1)).all()
    hold(out[lead + 150:lead + 350, :1], lse[lead + 150:lead + 350, :1], q[lead + 150:lead + 350, :1],
         k[lead + 150:lead + 350, :1], v[lead + 150:lead + 350, :1], OA.chain(200, 200), dim ** -0.5, dtype)


def test_prompt_sequences_do_not_depend_on_each_other(cuda):
    """Bits of a sequence alone and among others, call to call, and on another stream."""
    nq, dim = [40, 333, 1, 190], 128
    q, k, v = normal((sum(nq), 8, dim), "bf16", 30), normal((sum(nq), 2, dim), "bf16", 31), normal((sum(nq), 2, dim), "bf16", 32)
    cu = starts(nq)
    out, lse = run_prompt(q, k, v, cu, cu)
    again, _ = run_prompt(q, k, v, cu, cu)
    assert torch.equal(out, again)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o3, l3 = torch.zeros_like(out), torch.zeros_like(lse)
    side.wait_stream(torch.cuda.current_stream())
    A.moe_attention_prompt(q, k, v, cu, cu, o3, lse=l3, stream=side)
    side.synchronize()
    assert torch.equal(out, o3) and torch.equal(lse, l3)
    a = 0
    for n in nq:
        one, _ = run_prompt(q[a:a + n], k[a:a + n], v[a:a + n], starts([n]), starts([n]))
        assert torch.equal(one, out[a:a + n])
        a += n


def test_prompt_bad_offsets_stay_in_bounds(cuda):
    """Offsets past the tensors are cut to them; sequences that run backwards are empty."""
    q, k, v = normal((40, 2, 64), "bf16", 33), normal((40, 2, 64), "bf16", 34), normal((40, 2, 64), "bf16", 35)
    out, lse = run_prompt(q, k, v, ints([-5, 20, 10, 1000]), ints([0, 20, 500, 30]))
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()


# ------------------------------------------------------------------------------------------------------------------

def make_cache(lengths, kv, dim, page, dtype, seed, spare=3, poison=None, order=None, layers=2):
    """A cache of these sequences with pages anywhere; what no token owns holds `poison`."""
    held = [-(-n // page) for n in lengths]
    n_pages = sum(held) + spare
    g = torch.Generator().manual_seed(seed)
    pages = normal((2 * layers, n_pages, page, kv, dim), dtype, seed + 1)
    ids = torch.randperm(n_pages, generator=g).tolist() if order is None else order
    table = torch.full((len(lengths), max(max(held), 1) + 1), -1, dtype=torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32)
    at = 0
    owned = torch.zeros((n_pages, page), dtype=torch.bool)
    for s, (n, h) in enumerate(zip(lengths, held)):
        table[s, :h] = torch.tensor(ids[at:at + h], dtype=torch.int32)
        refs[ids[at:at + h]] = 1
        for p in range(n):
            owned[ids[at + p // page], p % page] = True
        at += h
    if poison is not None:
        pages[:, ~owned.cuda()] = poison
    return A.KVCache(pages, table.cuda(), ints(lengths), ints(held), refs.cuda())


def rows_of(cache, s, layer):
    n, page = int(cache.length[s]), cache.pages.shape[2]
    pages = cache.table[s, :-(-n // page)].long()
    return tuple(cache.pages[2 * layer + i][pages].flatten(0, 1)[:n] for i in (0, 1))


def run_cached(q, cache, layer, seqs, cu, mask=None, scale=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda")
    ws = A.cached_workspace(cache, seqs.numel(), q.shape[0], q.shape[1]).fill_(255)
    A.moe_attention_cached(q, cache, layer, seqs, cu, out, ws, mask=mask, lse=lse, scale=scale)
    torch.cuda.synchronize()
    return out, lse


def check_cached(lengths, draft, heads, kv, dim, page, dtype, seed=0, bits=None, words=None, poison=float("nan"), scale=None,
                 spread=1.0):
    """bits: per sequence the drafted tokens' mask [n, n], or None for a chain."""
    cache = make_cache(lengths, kv, dim, page, dtype, seed, poison=poison)
    order = np.random.RandomState(seed).permutation(len(lengths))
    draft = [draft[s] for s in order]
    q = normal((sum(draft), heads, dim), dtype, seed + 2, spread)
    mask = None
    if bits is not None:
        words = words or max(1, -(-max(draft) // 32))
        packed = np.zeros((sum(draft), words), dtype=np.uint32)
        at = 0
        for s, n in zip(order, draft):
            for i in range(n):
                for j in np.flatnonzero(bits[s][i]):
                    packed[at + i, j >> 5] |= np.uint32(1 << (j & 31))
            at += n
        mask = torch.from_numpy(packed.view(np.int32)).cuda()
    seqs = ints([int(s) for s in order])
    out, lse = run_cached(q, cache, 1, seqs, starts(draft), mask, scale)
    assert N.check_status() == 0
    at = 0
    for s, n in zip(order, draft):
        k, v = rows_of(cache, int(s), 1)
        seen = OA.chain(n, lengths[s]) if bits is None else OA.tree(bits[s], lengths[s])
        hold(out[at:at + n], lse[at:at + n], q[at:at + n], k, v, seen, dim ** -0.5 if scale is None else scale, dtype)
        at += n
    return out


@pytest.mark.parametrize("page", [1, 5, 16, 64, 200])
@pytest.mark.parametrize("dtype,heads,kv,dim", [("bf16", 8, 1, 128), ("fp16", 4, 4, 64), ("bf16", 14, 2, 80)])
def test_cached_single_tokens(cuda, page, dtype, heads, kv, dim):
    check_cached([1, 2, 15, 16, 17, 127, 128, 129, 300], [1] * 9, heads, kv, dim, page, dtype)


@pytest.mark.parametrize("length", [511, 1024, 2500, 5000, 9001])
@pytest.mark.parametrize("dtype,heads,kv,dim", [("bf16", 8, 2, 128), ("fp16", 2, 1, 64)])
def test_cached_long_sequences(cuda, length, dtype, heads, kv, dim):
    """Lengths that are worked on in pieces."""
    check_cached([length, 70, length // 2], [1, 3, 2], heads, kv, dim, 32, dtype, seed=40)


@pytest.mark.parametrize("draft", [[1, 2, 3], [17, 16, 0], [33, 64, 40], [130, 1, 129], [7, 300, 260]])
def test_cached_chains(cuda, draft):
    check_cached([700, 400, 260], draft, 4, 2, 64, 16, "bf16", seed=41)
    check_cached([700, 400, 260], draft, 7, 1, 128, 16, "fp16", seed=42)


@pytest.mark.parametrize("lengths,draft", [([5, 40, 300], [5, 40, 33]), ([200, 131, 1000], [64, 3, 12]), ([2000], [96])])
@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "fp16")])
def test_cached_trees(cuda, lengths, draft, dim, dtype):
    rng = np.random.RandomState(len(draft))
    parents = [[int(rng.randint(-1, j)) if j else -1 for j in range(n)] for n in draft]
    check_cached(lengths, draft, 8, 2, dim, 16, dtype, seed=43, bits=[OA.ancestors(p) for p in parents])


def test_cached_any_bits(cuda):
    """Bits that no tree has: nothing, everything, later tokens, not itself; rows that see nothing at all; too few words."""
    rng = np.random.RandomState(1)
    bits = [rng.rand(n, n) < 0.4 for n in (40, 40, 7, 35)]
    bits[1][:] = False
    bits[2][:] = True
    bits[3][:, 32:] = False  # what the words' own width leaves unseen
    check_cached([40, 40, 90, 500], [40, 40, 7, 35], 4, 1, 64, 8, "bf16", seed=44, bits=bits)
    check_cached([500], [35], 4, 1, 128, 8, "fp16", seed=45, bits=bits[3:], words=1)


def test_cached_more_queries_than_rows(cuda):
    check_cached([3, 0, 1], [9, 4, 1], 2, 1, 64, 4, "bf16", seed=46)
    check_cached([3, 0, 1], [9, 4, 1], 2, 1, 64, 4, "bf16", seed=47, bits=[np.ones((n, n), bool) for n in (9, 4, 1)])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_cached_sharp_scores(cuda, dtype):
    check_cached([3000, 200], [4, 20], 4, 1, 128, 64, dtype, seed=48, spread=20.0)


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_cached_poison_among_the_drafted(cuda, poison):
    """A drafted token's values reach its descendants alone."""
    lengths, n, dim = [600], 20, 64
    cache = make_cache(lengths, 1, dim, 16, "bf16", 50)
    page = int(cache.table[0, 595 // 16])
    cache.pages[1, page, 595 % 16, 0, 5] = poison       # values, drafted token 15
    cache.pages[0, int(cache.table[0, 598 // 16]), 598 % 16] = float("nan")  # keys, drafted token 18
    parents = [max(-1, j - 1 - j % 3) for j in range(n)]
    bits = OA.ancestors(parents)
    q = normal((n, 2, dim), "bf16", 51)
    mask = torch.zeros((n, 1), dtype=torch.int32, device="cuda")
    A.moe_tree_mask(ints(parents), ints([0, n]), mask)
    want = np.array([sum(1 << j for j in range(n) if bits[i, j]) for i in range(n)], dtype=np.int64).astype(np.int32)
    assert np.array_equal(mask[:, 0].cpu().numpy(), want)
    out, lse = run_cached(q, cache, 0, ints([0]), ints([0, n]), mask)
    k, v = rows_of(cache, 0, 0)
    clean = [i for i in range(n) if not bits[i, 18]]
    hold(out[clean], lse[clean], q[clean], k, v, OA.tree(bits, 600)[clean], dim ** -0.5, "bf16")
    assert torch.isnan(out[[i for i in range(n) if bits[i, 18]]].float()).all()


@pytest.mark.parametrize("n", [250, 256, 257, 600])
def test_cached_many_sequences(cuda, n):
    """Long ones, that are cut into pieces, among short ones, for more or fewer sequences than one plan holds."""
    rng = np.random.RandomState(n)
    lengths = [int(rng.randint(1024, 2200)) if x < 0.1 else int(rng.randint(1, 200)) for x in rng.rand(n)]
    draft = [int(min(length, d)) for length, d in zip(lengths, rng.randint(0, 4, n))]
    check_cached(lengths, draft, 2, 1, 64, 16, "bf16", seed=n)


def test_cached_sizes_of_many_classes(cuda):
    check_cached([33100, 40, 5000, 33000, 1], [1, 2, 40, 3, 1], 2, 1, 64, 64, "bf16", seed=9)


def test_prompt_thousands_of_sequences(cuda):
    rng = np.random.RandomState(1)
    nq = (rng.randint(1, 4, 8500) * (rng.rand(8500) < 0.1)).tolist()
    check_prompt(nq, nq, 2, 1, 64, "bf16", seed=11)


def test_prompt_sizes_of_one_call(cuda):
    """Many classes of sizes: prompts of 1 to 2000 tokens, with and without earlier keys."""
    nq = [1, 2000, 17, 900, 400, 400, 33, 1200, 5, 640]
    check_prompt(nq, [n + x for n, x in zip(nq, [0, 0, 700, 0, 300, 0, 1500, 0, 5, 0])], 4, 1, 64, "bf16", seed=12)


def test_cached_shared_pages_and_prompt_agree(cuda):
    """A prompt written into the cache (and a fork of it) gives what the packed form gives."""
    n, heads, kv, dim = 333, 8, 2, 128
    q, k, v = normal((n, heads, dim), "bf16", 52), normal((n, kv, dim), "bf16", 53), normal((n, kv, dim), "bf16", 54)
    cache = A.KVCache.empty(1, 40, 16, kv, dim, 4, 30)
    ws = A.pages_workspace(cache)
    A.moe_kv_extend(cache, ints([2]), ints([n]), ws)
    A.moe_kv_append(cache, 0, ints([2]), ints([0, n]), k, v)
    A.moe_kv_fork(cache, ints([2]), ints([0]))
    out, lse = run_prompt(q, k, v, ints([0, n]), ints([0, n]))
    for s in (2, 0):
        o, e = run_cached(q, cache, 0, ints([s]), ints([0, n]))
        hold(o, e, q, k, v, OA.chain(n, n), dim ** -0.5, "bf16")
    assert N.check_status() == 0


def test_cached_sequences_do_not_depend_on_each_other(cuda):
    lengths, draft = [3000, 20, 700, 5000], [1, 4, 9, 2]
    cache = make_cache(lengths, 2, 128, 16, "bf16", 55, poison=float("nan"))
    q = normal((sum(draft), 8, 128), "bf16", 56)
    out, lse = run_cached(q, cache, 0, ints([0, 1, 2, 3]), starts(draft))
    again, _ = run_cached(q, cache, 0, ints([0, 1, 2, 3]), starts(draft))
    assert torch.equal(out, again)
    a = 0
    for s, n in enumerate(draft):
        one, e = run_cached(q[a:a + n], cache, 0, ints([s]), ints([0, n]))
        assert torch.equal(one, out[a:a + n]) and torch.equal(e, lse[a:a + n])
        a += n


def test_cached_in_a_graph(cuda):
    """Captured once, replayed on other lengths: everything that depends on them is decided on the device."""
    cache = make_cache([900, 3000], 1, 64, 16, "bf16", 57, spare=10)
    q = normal((2, 4, 64), "bf16", 58)
    seqs, cu = ints([0, 1]), ints([0, 1, 2])
    out, ws = torch.empty_like(q), A.cached_workspace(cache, 2, 2, 4)
    A.moe_attention_cached(q, cache, 0, seqs, cu, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.moe_attention_cached(q, cache, 0, seqs, cu, out, ws)
    for lengths in ([900, 3000], [17, 2999], [1, 300]):
        cache.length.copy_(ints(lengths))
        graph.replay()
        torch.cuda.synchronize()
        for s in (0, 1):
            k, v = rows_of(cache, s, 0)
            want, _, spread, product = OA.attention(f64(q[s:s + 1]), f64(k), f64(v), OA.chain(1, lengths[s]), 0.125)
            tol, _ = OA.tolerance(want, np.zeros((1, 4)), spread, product, 64, lengths[s], "bf16", 6.0)
            assert (np.abs(f64(out[s:s + 1]) - want) <= tol).all()


def test_cached_bad_ids_are_reported_and_not_followed(cuda):
    cache = make_cache([100, 200, 50], 1, 64, 16, "bf16", 59)
    q = normal((4, 2, 64), "bf16", 60)
    assert N.check_status() == 0
    out, lse = run_cached(q, cache, 0, ints([0, 7, -1, 2]), ints([0, 1, 2, 3, 4]))
    assert N.check_status() == 1 and N.check_status() == 0
    assert (out[1:3] == 0).all() and torch.isinf(lse[1:3]).all()
    for i, s in ((0, 0), (3, 2)):
        k, v = rows_of(cache, s, 0)
        hold(out[i:i + 1], lse[i:i + 1], q[i:i + 1], k, v, OA.chain(1, k.shape[0]), 0.125, "bf16")
    cache.table[1, 3] = 10 ** 6
    cache.table[2, 0] = -7
    cache.length[0] = 10 ** 8
    run_cached(q[:3], cache, 0, ints([0, 1, 2]), ints([0, 1, 2, 3]))
    assert N.check_status() == 1


def test_cached_offsets_past_32_bits(cuda):
    """Pages whose elements lie past 2^31 (and bytes past 2^32)."""
    page, kv, dim = 64, 8, 128
    n_pages = (1 << 31) // (page * kv * dim) + 40
    pages = torch.empty((2, n_pages, page, kv, dim), dtype=torch.bfloat16, device="cuda")
    ids = [n_pages - 1, 3, n_pages - 2, n_pages // 2, n_pages - 5, n_pages - 9]
    for i, p in enumerate(ids):
        pages[:, p] = normal((2, page, kv, dim), "bf16", 61 + i)
    table = torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    table[0, :6] = ints(ids)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[torch.tensor(ids, device="cuda")] = 1
    cache = A.KVCache(pages, table, ints([370]), ints([6]), refs)
    q = normal((3, 16, dim), "bf16", 70)
    out, lse = run_cached(q, cache, 0, ints([0]), ints([0, 3]))
    k, v = rows_of(cache, 0, 0)
    hold(out, lse, q, k, v, OA.chain(3, 370), dim ** -0.5, "bf16")
    assert N.check_status() == 0


def test_binding_refusals(cuda):
    cache = A.KVCache.empty(1, 4, 16, 2, 64, 2, 4)
    q, cu, seqs = normal((3, 4, 64), "bf16", 71), ints([0, 3]), ints([0])
    out, ws = torch.empty_like(q), A.cached_workspace(cache, 1, 3, 4)
    kv = normal((3, 2, 64), "bf16", 72)
    for bad in (lambda: A.moe_attention_cached(q.half(), cache, 0, seqs, cu, out.half(), ws),
                lambda: A.moe_attention_cached(q, cache, 0, seqs.long(), cu, out, ws),
                lambda: A.moe_attention_cached(q, cache, 0, seqs, ints([0, 1, 3]), out, ws),
                lambda: A.moe_attention_cached(q, cache, 0, seqs, cu, out[:2], ws),
                lambda: A.moe_attention_cached(q[..., :32], cache, 0, seqs, cu, out[..., :32], ws),
                lambda: A.moe_attention_prompt(q.float(), kv, kv, cu, cu, out),
                lambda: A.moe_attention_prompt(q, kv.half(), kv, cu, cu, out),
                lambda: A.moe_attention_prompt(q.transpose(1, 2), kv, kv, cu, cu, out),
                lambda: A.moe_attention_prompt(q, kv, kv, cu.cpu(), cu, out),
                lambda: A.moe_attention_prompt(q, kv, kv, cu, cu, out, lse=torch.empty(3, 4, dtype=torch.float64, device="cuda")),
                lambda: A.KVCache(cache.pages, cache.table, cache.length, cache.held, cache.refs[:-1]),
                lambda: A.KVCache(cache.pages.float(), cache.table, cache.length, cache.held, cache.refs),
                lambda: A.moe_kv_append(cache, 0, seqs, cu, kv[:, :1], kv)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError, match="invalid argument"):
        A.moe_attention_cached(q, cache, 1, seqs, cu, out, ws)
    with pytest.raises(RuntimeError, match="unsupported shape"):
        A.moe_attention_cached(normal((3, 5, 64), "bf16", 73), cache, 0, seqs, cu, torch.empty((3, 5, 64), dtype=torch.bfloat16,
                                                                                              device="cuda"), ws)


@pytest.mark.parametrize("sizes,words", [([1, 2, 33, 0, 64, 31], 2), ([256, 255], 8), ([300, 5], 11), ([7], 3)])
def test_tree_masks(cuda, sizes, words):
    """Ancestors' bits in every word of the rows, for trees that fit one CTA's table and one that does not; a chain
    (the longest walk) among them."""
    rng = np.random.RandomState(len(sizes))
    parents = [[j - 1 for j in range(n)] if i == 0 else [int(rng.randint(-1, j)) if j else -1 for j in range(n)]
               for i, n in enumerate(sizes)]
    mask = torch.full((sum(sizes), words), 77, dtype=torch.int32, device="cuda")
    A.moe_tree_mask(ints(sum(parents, [])), starts(sizes), mask)
    got, at = mask.cpu().numpy().view(np.uint32), 0
    for p in parents:
        bits = OA.ancestors(p)
        for i in range(len(p)):
            row = [(got[at + i, j >> 5] >> (j & 31)) & 1 for j in range(32 * words)]
            assert row[:len(p)] == bits[i].astype(int).tolist() and not any(row[len(p):]), (len(p), i)
        at += len(p)
    assert N.check_status() == 0


def test_tree_mask_bad_parents_and_words(cuda):
    mask = torch.full((5, 1), 77, dtype=torch.int32, device="cuda")
    A.moe_tree_mask(ints([-1, 0, 2, -5, 1]), ints([0, 5]), mask)
    assert mask[:, 0].tolist() == [1, 3, 4, 8, 19] and N.check_status() == 1
    mask = torch.full((40, 1), 77, dtype=torch.int32, device="cuda")
    A.moe_tree_mask(ints(list(range(-1, 33)) + [-1] * 6), ints([0, 34, 40]), mask)
    assert mask[:, 0].tolist() == [0] * 34 + [1 << j for j in range(6)] and N.check_status() == 1
