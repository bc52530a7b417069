"""The attention operators' C ABI without a GPU: the library exports what the
header declares, and bad arguments are refused on the host before any CUDA
call. And the definitions that the GPU tests hold the kernels to."""
import ctypes
import os
import re

import numpy as np
import pytest

from nvfp4_block_scaled_gather_gb300 import attention as A
from oracle import attention as OA
from oracle.kv_pages import Pages
from tests.conftest import ROOT

INVALID, SHAPE, WORKSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def lib(native):
    return A.load()


def cache(**other):
    """A cache of made-up aligned addresses: nothing here reaches the device."""
    c = dict(pages=4096, planes=4, n_pages=8, page_size=16, heads_kv=2, head_dim=64, dtype=0, table=4096, length=4096,
             held=4096, refs=4096, max_seqs=4, max_pages=4)
    c.update(other)
    return ctypes.byref(A.CacheStruct(*[c[n] for n, _ in A.CacheStruct._fields_]))


def heads(data=4096, ts=256, hs=64):
    return ctypes.byref(A.Heads(data, ts, hs))


def test_library_exports_every_declared_symbol(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_attention.h")).read(), flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", src, flags=re.M)
    assert set(names) == set(A.exported_symbols())
    for n in names:
        assert hasattr(lib, n), n
    assert lib.moe_nvfp4_error_string(6) == b"out of cache pages"


@pytest.mark.parametrize("other,status", [
    (dict(pages=0), INVALID), (dict(pages=4104), INVALID), (dict(table=0), INVALID), (dict(refs=4104), INVALID),
    (dict(planes=0), INVALID), (dict(planes=3), SHAPE), (dict(n_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(heads_kv=0), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=60), SHAPE), (dict(dtype=2), INVALID),
    (dict(max_seqs=0), INVALID), (dict(max_pages=-1), INVALID), (dict(n_pages=1 << 20, page_size=1 << 12), SHAPE),
])
def test_bad_caches_are_refused_everywhere(lib, other, status):
    c = cache(**other)
    assert lib.moe_kv_workspace_size(c) == 0
    assert lib.moe_kv_extend(c, 16, 16, 1, 256, 1 << 20, None) == status
    assert lib.moe_kv_append(c, 0, 16, 16, 1, 1, heads(), heads(), None) == status
    assert lib.moe_kv_fork(c, 16, 16, 1, None) == status
    assert lib.moe_kv_truncate(c, 16, 16, 1, None) == status
    assert lib.moe_kv_keep(c, 16, 16, 16, 1, 16, 1, 256, 1 << 20, None) == status
    assert lib.moe_kv_copy_pages(c, 16, 16, 1, None) == status
    assert lib.moe_kv_compact(c, 256, 1 << 20, None) == status
    assert lib.moe_attention_cached_workspace_size(c, 1, 1, 4) == 0
    assert lib.moe_attention_cached(heads(), c, 0, 16, 16, 1, 1, 4, None, 0, 0.1, heads(), None, 256, 1 << 30,
                                    None) == status


def test_pages_refusals(lib):
    c = cache()
    size = lib.moe_kv_workspace_size(c)
    assert size > 0
    assert lib.moe_kv_extend(c, 16, 16, 1, 256, size - 1, None) == WORKSPACE
    assert lib.moe_kv_extend(c, 16, 16, 1, 300, size, None) == INVALID
    assert lib.moe_kv_extend(c, None, 16, 1, 256, size, None) == INVALID
    assert lib.moe_kv_extend(c, 16, 16, -1, 256, size, None) == INVALID
    assert lib.moe_kv_extend(c, 16, 16, 5, 256, size, None) == INVALID      # more than there are sequences
    assert lib.moe_kv_truncate(c, 16, 16, 4097, None) == INVALID
    assert lib.moe_kv_truncate(c, 16, None, 1, None) == INVALID
    assert lib.moe_kv_fork(c, None, 16, 1, None) == INVALID
    assert lib.moe_kv_append(c, 2, 16, 16, 1, 1, heads(), heads(), None) == INVALID
    assert lib.moe_kv_append(c, -1, 16, 16, 1, 1, heads(), heads(), None) == INVALID
    assert lib.moe_kv_append(c, 0, 16, 16, 1, 1, heads(4100), heads(), None) == INVALID
    assert lib.moe_kv_append(c, 0, 16, 16, 1, 1, heads(), heads(ts=100), None) == INVALID
    assert lib.moe_kv_append(c, 0, 16, 16, 1, 1, None, heads(), None) == INVALID
    assert lib.moe_kv_keep(c, 16, 16, None, 1, 16, 1, 256, size, None) == INVALID
    assert lib.moe_kv_keep(c, 16, 16, 16, -1, 16, 1, 256, size, None) == INVALID
    assert lib.moe_kv_keep(c, 16, 16, 16, 1, 16, 1, 256, 16, None) == WORKSPACE
    assert lib.moe_kv_copy_pages(c, 16, None, 1, None) == INVALID
    assert lib.moe_kv_compact(c, None, size, None) == INVALID
    assert lib.moe_kv_compact(c, 256, size - 1, None) == WORKSPACE
    assert lib.moe_tree_mask(16, 16, 1, 4, 16, 0, None) == INVALID
    assert lib.moe_tree_mask(None, 16, 1, 4, 16, 1, None) == INVALID
    # nothing to do
    assert lib.moe_kv_extend(c, None, None, 0, None, 0, None) == 0
    assert lib.moe_kv_append(c, 0, None, None, 0, 0, None, None, None) == 0
    assert lib.moe_kv_truncate(c, None, None, 0, None) == 0
    assert lib.moe_kv_fork(c, None, None, 0, None) == 0
    assert lib.moe_kv_keep(c, None, None, None, 0, None, 0, None, 0, None) == 0
    assert lib.moe_kv_copy_pages(c, None, None, 0, None) == 0
    assert lib.moe_tree_mask(None, None, 0, 0, None, 1, None) == 0


def test_attention_refusals(lib):
    def prompt(q=heads(), k=heads(), v=heads(), cu_q=16, cu_k=16, n=1, tq=4, tk=4, hq=4, hkv=2, d=64, dtype=0,
               scale=0.1, out=heads(), lse=None):
        return lib.moe_attention_prompt(q, k, v, cu_q, cu_k, n, tq, tk, hq, hkv, d, dtype, scale, out, lse, None)

    for bad in (dict(q=None), dict(out=None), dict(k=heads(0)), dict(q=heads(4100)), dict(v=heads(hs=4)),
                dict(q=heads(ts=-8)), dict(cu_q=None), dict(cu_k=None), dict(n=-1), dict(tq=-1), dict(tk=-1),
                dict(hq=0), dict(hkv=0), dict(d=0), dict(dtype=3), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert prompt(**bad) == INVALID, bad
    for bad in (dict(d=60), dict(d=136), dict(hq=5), dict(hq=258, hkv=2), dict(tq=1 << 30)):
        assert prompt(**bad) == SHAPE, bad
    assert prompt(n=0) == 0 and prompt(tq=0) == 0

    c = cache()
    size = lib.moe_attention_cached_workspace_size(c, 1, 1, 4)

    def cached(q=heads(), cache_=c, layer=0, seqs=16, cu_q=16, n=1, tq=1, hq=4, mask=None, words=0, scale=0.1,
               out=heads(), ws=256, ws_bytes=size):
        return lib.moe_attention_cached(q, cache_, layer, seqs, cu_q, n, tq, hq, mask, words, scale, out, None, ws,
                                        ws_bytes, None)

    for bad in (dict(q=None), dict(out=heads(4100)), dict(cache_=None), dict(layer=2), dict(layer=-1), dict(seqs=None),
                dict(cu_q=None), dict(n=-1), dict(tq=-1), dict(hq=0), dict(mask=16, words=0), dict(words=-1),
                dict(scale=0.0), dict(ws=None), dict(ws=300)):
        assert cached(**bad) == INVALID, bad
    assert cached(hq=3) == SHAPE
    assert cached(cache_=cache(head_dim=136)) == SHAPE
    assert cached(ws_bytes=size - 1) == WORKSPACE
    assert cached(n=0) == 0 and cached(tq=0) == 0


def test_definition_of_attention():
    """The oracle against the formula written out for two keys, and its masks."""
    q, k, v = np.array([[[2.0]]]), np.array([[[1.0]], [[3.0]]]), np.array([[[10.0]], [[20.0]]])
    out, lse, _, _ = OA.attention(q, k, v, np.ones((1, 2), bool), 0.5)
    w = np.exp([1.0, 3.0])
    assert np.isclose(out[0, 0, 0], (w @ [10.0, 20.0]) / w.sum()) and np.isclose(lse[0, 0], np.log(w.sum()))
    out, lse, _, _ = OA.attention(q, k, v, np.zeros((1, 2), bool), 0.5)
    assert out[0, 0, 0] == 0 and lse[0, 0] == -np.inf
    assert OA.chain(2, 3).tolist() == [[True, True, False], [True, True, True]]
    assert OA.chain(3, 2).tolist() == [[False, False], [True, False], [True, True]]
    assert OA.ancestors([-1, 0, 0, 1]).astype(int).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 1, 0, 1]]
    assert OA.tree(np.eye(2, dtype=bool), 3).tolist() == [[True, True, False], [True, False, True]]


def test_definition_of_pages():
    p = Pages(6, 4, 3, 4)
    assert p.extend([0], [6]) is True and p.table[0] == [0, 1]
    for pos in range(6):
        p.write(0, pos, pos)
    p.fork(0, 2)
    assert p.refs[:2] == [2, 2]
    assert p.extend([0, 2], [1, 1]) is True            # the first to grow leaves the shared open page, the second stays
    assert p.table[0] == [0, 2] and p.table[2] == [0, 1] and p.refs[:3] == [2, 1, 1]
    assert [p.read(0, i) for i in range(6)] == list(range(6))
    assert p.extend([1], [17]) is False and p.extend([1], [16]) == "pages"
    p.truncate(0, 0)
    assert p.refs == [1, 1, 0, 0, 0, 0]
    p.extend([1], [4])
    p.truncate(2, 0)
    assert p.table[1] == [2]
    p.compact()
    assert p.table[1] == [0] and p.refs == [1, 0, 0, 0, 0, 0]
