"""Upkeep of the paged cache against its definition (oracle.kv_pages): every
table, count and row after every step."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_gather_gb300 import _native as N
from nvfp4_block_scaled_gather_gb300 import attention as A
from oracle.kv_pages import Pages

pytestmark = pytest.mark.gpu
INVALID, OUT_OF_PAGES = 1, 6


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Both:
    """The library's cache and the definition's, driven together. A row's value is its number: the library's rows
    hold it in every plane, offset by the plane."""

    def __init__(self, n_pages, page, max_seqs, max_pages, kv=2, dim=8, layers=2, dtype=torch.bfloat16):
        self.cache = A.KVCache.empty(layers, n_pages, page, kv, dim, max_seqs, max_pages, dtype=dtype)
        self.model = Pages(n_pages, page, max_seqs, max_pages)
        self.ws = A.pages_workspace(self.cache).fill_(255)
        self.next = 1
        assert N.check_status() == 0

    def bits(self, value, plane):
        return (value * 7 + plane * 1009) % 30000 + 1  # as int16 patterns

    def check(self, status=0):
        torch.cuda.synchronize()
        assert N.check_status() == status
        c, m = self.cache, self.model
        assert c.length.tolist() == m.length
        assert c.held.tolist() == [len(t) for t in m.table]
        assert c.refs.tolist() == m.refs
        width = c.table.shape[1]
        assert c.table.tolist() == [t + [-1] * (width - len(t)) for t in m.table]
        got = c.pages.view(torch.int16)[..., 0, 0].cpu().numpy()
        whole = c.pages.view(torch.int16)
        assert bool((whole == whole[..., :1, :1]).all())  # a row's heads and elements move together
        for p, rows in enumerate(m.rows):
            for r, value in enumerate(rows):
                for plane in range(got.shape[0]):
                    want = 0 if value is None else self.bits(value, plane)
                    assert got[plane, p, r] == want, (plane, p, r)

    def extend(self, seqs, add, status=0):
        done = self.model.extend(seqs, add)
        assert (done is True) == (status == 0)
        A.moe_kv_extend(self.cache, ints(seqs), ints(add), self.ws)
        self.check(status)

    def append(self, seqs, counts, status=0):
        """New values for the last tokens, in every layer."""
        c, total = self.cache, sum(counts)
        numbers = list(range(self.next, self.next + total))
        self.next += total
        cu = ints(np.concatenate([[0], np.cumsum(counts)]).tolist())
        for layer in range(c.layers):
            k, v = (torch.tensor([self.bits(x, 2 * layer + i) for x in numbers], dtype=torch.int16, device="cuda")
                    .view(c.pages.dtype)[:, None, None].expand(total, c.pages.shape[3], c.pages.shape[4]).contiguous()
                    for i in (0, 1))
            A.moe_kv_append(c, layer, ints(seqs), cu, k, v)
        at = 0
        for s, n in zip(seqs, counts):
            for j in range(n):
                pos = self.model.length[s] - n + j
                if pos >= 0:
                    self.model.write(s, pos, numbers[at + j])
            at += n
        self.check(status)

    def grow(self, seqs, add):
        self.extend(seqs, add)
        self.append(seqs, add)

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            self.model.fork(a, b)
        A.moe_kv_fork(self.cache, ints(src), ints(dst))
        self.check()

    def truncate(self, seqs, to):
        for s, n in zip(seqs, to):
            self.model.truncate(s, n)
        A.moe_kv_truncate(self.cache, ints(seqs), ints(to))
        self.check()

    def keep(self, seqs, drafted, places, status=0, width=None):
        for s, n, at in zip(seqs, drafted, places):
            self.model.keep(s, n, at)
        width = width or max([len(p) for p in places] + [1])
        rows = [p + [99] * (width - len(p)) for p in places]
        A.moe_kv_keep(self.cache, ints(seqs), ints(drafted), ints(rows), ints([len(p) for p in places]), self.ws)
        self.check(status)

    def compact(self):
        self.model.compact()
        A.moe_kv_compact(self.cache, self.ws)
        self.check()


@pytest.mark.parametrize("page", [1, 3, 16])
def test_grow_write_and_free(cuda, page):
    b = Both(60, page, 5, 40)
    b.grow([3], [1])
    b.grow([0, 3, 4], [7, 0, 17])
    b.grow([4, 0], [1, 3])
    b.truncate([0, 4], [6, 100])
    b.truncate([3, 1], [0, 0])
    b.grow([1, 0], [5, 2])
    b.truncate([0, 1, 4], [0, 0, 0])
    assert not any(b.model.refs)


def test_forks_share_pages_until_they_grow(cuda):
    b = Both(40, 4, 8, 9)
    b.grow([0], [10])
    b.fork([0, 0, 0], [1, 2, 5])
    b.grow([1, 2, 5], [1, 1, 3])     # three copies of the open page
    b.grow([0], [1])                 # the last holder writes in place
    b.fork([1], [3])
    b.truncate([3], [5])             # ends inside a page that others hold as a full one
    b.grow([3, 1], [2, 4])
    b.fork([2, 2], [4, 6])
    b.grow([6, 2, 4], [1, 1, 1])     # all holders of a page at once: the last of them keeps it
    b.truncate([0, 1, 2, 3, 4, 5, 6], [0] * 7)
    assert not any(b.model.refs)


@pytest.mark.parametrize("page,kv,dim", [(64, 8, 128), (37, 3, 120), (5, 16, 128)])
def test_copies_of_large_pages(cuda, page, kv, dim):
    """Pages of several units of copying (128 KB), of one and a half, and of a little more than one; part of them in use."""
    b = Both(90, page, 40, 8, kv=kv, dim=dim)
    b.grow([0, 30], [2 * page + page // 2, page + 1])
    b.fork([0] * 20, list(range(1, 21)))
    b.grow(list(range(1, 21)), [1 + i % 3 for i in range(20)])
    b.fork([30, 30], [31, 32])
    b.grow([32, 30, 31], [page, 1, 2])
    b.truncate([0, 3, 7, 30], [0, 0, page + 1, 0])
    b.compact()
    b.keep([5, 31], [2, 1], [[1], []])
    b.truncate(list(range(1, 21)), [0] * 20)
    b.compact()


def test_forks_of_empty_and_whole_page_sequences(cuda):
    b = Both(20, 4, 6, 5)
    b.grow([0], [8])
    b.fork([0, 4], [1, 2])
    b.grow([1, 2], [1, 1])


@pytest.mark.parametrize("page", [1, 4, 7])
def test_keep_moves_rows_together(cuda, page):
    b = Both(60, page, 4, 30, kv=3, dim=40)
    b.grow([0, 1, 2], [5, 11, 0])
    b.grow([0, 1, 2], [9, 6, 20])
    b.keep([2, 0, 1], [20, 9, 6], [[0, 1, 5, 6, 13, 19], [], [0, 1, 2, 3, 4, 5]])
    b.grow([0, 1, 2], [3, 3, 3])
    b.keep([1, 0], [3, 3], [[2], [0, 2]], width=7)
    b.keep([2], [0], [[]])


def test_keep_of_many_rows(cuda):
    """More kept rows than one pass of a CTA's table takes, and rows of more than one CTA's bytes."""
    b = Both(40, 16, 2, 40, kv=9, dim=128, layers=1)
    b.grow([1], [13])
    b.grow([1], [400])
    b.keep([1], [400], [sorted(np.random.RandomState(0).choice(400, 290, replace=False).tolist())])


def test_compaction(cuda):
    b = Both(64, 4, 8, 12)
    for s in range(8):
        b.grow([s], [5 + 4 * s])
    b.fork([7], [0]) if not b.model.length[0] else None
    b.truncate([0, 2, 5], [0, 0, 3])
    b.fork([6], [2])
    b.compact()
    b.compact()                       # nothing left to move
    b.grow([0, 2], [9, 1])
    b.truncate(list(range(8)), [0] * 8)
    b.compact()


def test_compaction_of_a_large_pool(cuda):
    """Several pages to a thread of the plan."""
    b = Both(5000, 2, 6, 2000, kv=1, layers=1)
    b.extend([0, 1, 2, 3], [1000, 3001, 500, 3999])
    b.truncate([1, 0], [7, 998])
    b.compact()
    b.extend([4, 1], [2500, 301])


def test_copy_pages(cuda):
    b = Both(12, 4, 3, 6)
    b.grow([0], [13])
    for s, d in ((0, 7), (2, 9), (3, 11)):
        b.model.rows[d] = list(b.model.rows[s])
    A.moe_kv_copy_pages(b.cache, ints([0, 2, 3, 5]), ints([7, 9, 11, 5]))
    b.check()
    A.moe_kv_copy_pages(b.cache, ints([0, 99, 1]), ints([12, 1, -1]))
    b.check(INVALID)


def test_too_few_pages_changes_nothing(cuda):
    b = Both(6, 4, 4, 6)
    b.grow([0], [9])
    b.fork([0], [1])
    b.extend([1, 2], [1, 12], status=OUT_OF_PAGES)  # one copy and three pages, three are free
    b.grow([1, 2], [1, 8])
    b.extend([3], [1], status=OUT_OF_PAGES)
    b.truncate([2], [0])
    b.grow([3], [1])


def test_bad_arguments_are_reported_and_left_alone(cuda):
    b = Both(16, 4, 4, 4)
    b.grow([0, 1], [6, 9])
    b.extend([0, 0], [1, 1], status=INVALID)
    b.extend([2], [17], status=INVALID)             # more than max_pages
    for seqs, add in (([4], [1]), ([-1], [1]), ([2], [-1])):
        A.moe_kv_extend(b.cache, ints(seqs), ints(add), b.ws)
        b.check(INVALID)
    for src, dst in (([0], [1]), ([0], [0]), ([9], [2]), ([0], [-1]), ([0, 2], [2, 3])):
        A.moe_kv_fork(b.cache, ints(src), ints(dst))
        if (src, dst) == ([0, 2], [2, 3]):
            b.model.fork(2, 3)                       # the second pair is a good one: both are empty
        b.check(INVALID)
    A.moe_kv_fork(b.cache, ints([0, 1]), ints([2, 2]))
    b.model.fork(0, 2)                               # a repeated dst goes to its first pair
    b.check(INVALID)
    for seqs, to in (([4], [1]), ([-3], [1]), ([1], [-1])):
        A.moe_kv_truncate(b.cache, ints(seqs), ints(to))
        b.check(INVALID)
    # keep: not ascending, past the drafted, more drafted than there are, more kept than drafted; and a shared page
    for drafted, keep, kept in ((3, [1, 1], 2), (3, [0, 3], 2), (10, [0, 1], 2), (1, [0, 1], 2), (3, [-1, 0], 2)):
        A.moe_kv_keep(b.cache, ints([1]), ints([drafted]), ints([keep]), ints([kept]), b.ws)
        b.check(INVALID)
    b.keep([2], [2], [[1]], status=INVALID)
    # append into a shared page
    b.append([2], [2], status=INVALID)
    # ... and one more row than the sequence has
    b.append([1], [10], status=INVALID)


@pytest.mark.parametrize("seed", range(4))
def test_random_steps(cuda, seed):
    rng = np.random.RandomState(seed)
    page = int(rng.choice([2, 4, 16]))
    b = Both(50, page, 7, 12, kv=int(rng.randint(1, 4)), dim=int(rng.choice([8, 64])), layers=int(rng.randint(1, 3)))
    for _ in range(25):
        m = b.model
        live = [s for s in range(7) if m.length[s]]
        what = rng.choice(["grow", "fork", "truncate", "keep", "compact"], p=[0.4, 0.2, 0.15, 0.2, 0.05])
        if what == "grow":
            seqs = rng.permutation(7)[:rng.randint(1, 5)].tolist()
            add = [int(rng.randint(0, max(1, min(2 * page, 12 * page - m.length[s]) + 1))) for s in seqs]
            trial = Pages.__new__(Pages)
            trial.__dict__ = {k: ([list(r) if isinstance(r, list) else r for r in v] if isinstance(v, list) else v)
                              for k, v in m.__dict__.items()}
            if trial.extend(seqs, add) is True:
                b.grow(seqs, add)
            else:
                b.extend(seqs, add, status=OUT_OF_PAGES)
        elif what == "fork" and live and len(live) < 7:
            dst = [s for s in range(7) if s not in live]
            dst = rng.permutation(dst)[:rng.randint(1, len(dst) + 1)].tolist()
            b.fork(rng.choice(live, len(dst)).tolist(), dst)
        elif what == "truncate" and live:
            seqs = rng.permutation(live)[:2].tolist()
            b.truncate(seqs, [int(rng.randint(0, m.length[s] + 2)) for s in seqs])
        elif what == "keep" and live:
            s = int(rng.choice(live))
            n = int(rng.randint(0, m.length[s] + 1))
            at = sorted(rng.permutation(n)[:rng.randint(0, n + 1)].tolist())
            shared = at and any(m.refs[p] != 1 for p in m.table[s][(m.length[s] - n) // page:])
            b.keep([s], [n], [at], status=INVALID if shared else 0)
        elif what == "compact":
            b.compact()


def test_many_sequences_at_once(cuda):
    """More sequences than the plan has threads."""
    b = Both(4000, 2, 1500, 4, kv=1, layers=1)
    rng = np.random.RandomState(5)
    order = rng.permutation(1500).tolist()
    b.extend(order, rng.randint(0, 5, 1500).tolist())
    b.extend(order[:1100], rng.randint(0, 3, 1100).tolist())


def test_offsets_past_32_bits(cuda):
    """Copies to and from pages whose bytes lie past 2^32, and planes beyond them."""
    page, kv, dim = 256, 8, 128
    n_pages = (1 << 32) // (page * kv * dim * 2) + 8
    cache = A.KVCache.empty(1, n_pages, page, kv, dim, 2, n_pages)
    cache.pages[:, n_pages - 1] = torch.randn((2, page, kv, dim), device="cuda").bfloat16()
    cache.pages[:, 2] = torch.randn((2, page, kv, dim), device="cuda").bfloat16()
    A.moe_kv_copy_pages(cache, ints([n_pages - 1, 2]), ints([1, n_pages - 3]))
    assert torch.equal(cache.pages[:, 1], cache.pages[:, n_pages - 1])
    assert torch.equal(cache.pages[:, 2], cache.pages[:, n_pages - 3]) and bool(cache.pages[1, 2].any())
    cache.refs[n_pages - 1] = 1
    cache.table[1, 0], cache.held[1], cache.length[1] = n_pages - 1, 1, 9
    want = cache.pages[:, n_pages - 1].clone()
    A.moe_kv_compact(cache, A.pages_workspace(cache))
    assert cache.table[1, 0].item() == 0 and torch.equal(cache.pages[:, 0], want)
    assert N.check_status() == 0
