"""The cache-and-attention operators of the library: what is measured, and their plain forms.

Three operators that a serving engine runs next to the routed-expert layer:

  prompt   causal attention over whole prompts, grouped heads, packed sequences of different lengths
  cached   attention of drafted tokens (a tree, or one token a stream) over a paged cache of keys and values
  pages    upkeep of that cache's pages: a draft step (grow, write, keep the accepted rows), forking with
           copy on growth, and compaction of the pool

`run` with own = False computes them by elementary torch operations in 32 bits; with own = True it calls the
library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one short chat turn entering an idle engine: latency
        dict(name="prompt_turn", op="prompt", dtype="bf16", seqs=1, lo=23, hi=23, past=0, heads=32, kv_heads=4, dim=128),
        # a prefill batch of ragged prompts, grouped heads
        dict(name="prompt_ragged", op="prompt", dtype="bf16", seqs=9, lo=37, hi=1500, past=0, heads=32, kv_heads=4, dim=128),
        # the next pieces of long prompts, whose earlier keys are at hand: queries fewer than keys; 64-wide heads, no groups
        dict(name="prompt_pieces", op="prompt", dtype="fp16", seqs=5, lo=301, hi=1024, past=777, heads=16, kv_heads=16, dim=64),
        # one long document
        dict(name="prompt_document", op="prompt", dtype="bf16", seqs=1, lo=8192, hi=8192, past=0, heads=32, kv_heads=8, dim=128),
        # one stream, one token, a short conversation: latency
        dict(name="decode_one", op="cached", dtype="bf16", seqs=1, lo=700, hi=700, draft_lo=1, draft_hi=1, heads=32, kv_heads=4,
             dim=128, page=64),
        # the engine's usual decode batch
        dict(name="decode_batch", op="cached", dtype="bf16", seqs=32, lo=500, hi=6000, draft_lo=1, draft_hi=1, heads=32,
             kv_heads=8, dim=128, page=64),
        # drafted trees of different sizes over middling contexts, small pages
        dict(name="tree_batch", op="cached", dtype="fp16", seqs=16, lo=300, hi=5000, draft_lo=5, draft_hi=24, heads=32,
             kv_heads=4, dim=128, page=16),
        # a large tree over long contexts
        dict(name="tree_long", op="cached", dtype="bf16", seqs=4, lo=24000, hi=40000, draft_lo=48, draft_hi=64, heads=32,
             kv_heads=8, dim=128, page=128),
        # a draft step of one stream: latency
        dict(name="step_one", op="pages", kind="step", dtype="bf16", seqs=1, lo=300, hi=300, draft_lo=8, draft_hi=8, layers=4,
             kv_heads=4, dim=128, page=16),
        # draft steps of a batch in a deep model's cache
        dict(name="step_batch", op="pages", kind="step", dtype="bf16", seqs=32, lo=100, hi=700, draft_lo=6, draft_hi=24,
             layers=16, kv_heads=8, dim=128, page=64),
        # several answers to each of some prompts: shared pages, the open one copied when the answers grow
        dict(name="fork_batch", op="pages", kind="fork", dtype="bf16", seqs=24, children=4, lo=70, hi=500, layers=16, kv_heads=8,
             dim=128, page=64),
        # half of the pool's sequences have ended: the others' pages move to the front
        dict(name="compact_pool", op="pages", kind="compact", dtype="bf16", seqs=24, lo=200, hi=600, layers=16, kv_heads=8,
             dim=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "cached", "pages"])
    dtype = rng.choice(["bf16", "fp16"])
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128, 128, 80])
    group = rng.choice([1, 2, 4, 7, 8])
    if op == "prompt":
        seqs = _log(rng, 1, 24)
        hi = _log(rng, 1, int(4400 / seqs ** 0.5))
        return dict(op=op, dtype=dtype, seqs=seqs, lo=_log(rng, 1, hi), hi=hi, past=rng.choice([0, 0, _log(rng, 1, 1 + hi // 3)]),
                    heads=kv * group, kv_heads=kv, dim=dim)
    if op == "cached":
        seqs = _log(rng, 1, 64)
        hi = _log(rng, 1, 90000 // seqs)
        draft = rng.choice([1, 1, _log(rng, 1, 64)])
        return dict(op=op, dtype=dtype, seqs=seqs, lo=_log(rng, 1, hi), hi=hi, draft_lo=_log(rng, 1, draft), draft_hi=draft,
                    heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64, 128]))
    kind = rng.choice(["step", "fork", "compact"])
    seqs = _log(rng, 1, 24)
    hi = _log(rng, 2, 600)
    case = dict(op=op, kind=kind, dtype=dtype, seqs=seqs, lo=_log(rng, 1, hi), hi=hi, layers=_log(rng, 1, 16), kv_heads=kv, dim=dim,
                page=rng.choice([16, 32, 64]))
    if kind == "step":
        draft = _log(rng, 1, 24)
        case.update(draft_lo=_log(rng, 1, draft), draft_hi=draft)
    if kind == "fork":
        case.update(children=rng.randint(1, 4))
    if kind == "compact":
        case.update(seqs=max(2, seqs))
    return case


def _lengths(lo, hi, n, salt):
    """n lengths in [lo, hi], both ends among them: a fixed spread that depends on the case alone."""
    return [hi if i == 0 else lo if i == 1 else lo + (i * 7919 + salt * 104729) % (hi - lo + 1) for i in range(n)]


def _prompt_lengths(case):
    nq = _lengths(case["lo"], case["hi"], case["seqs"], 1)
    return nq, [n + (case["past"] and 1 + (i * 389) % case["past"]) for i, n in enumerate(nq)]


def _cached_lengths(case):
    context = _lengths(case["lo"], case["hi"], case["seqs"], 2)
    draft = _lengths(case["draft_lo"], case["draft_hi"], case["seqs"], 3)
    return [c + d for c, d in zip(context, draft)], draft


# --------------------------------------------------------------------------------------------------------------
# the inputs
# --------------------------------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _starts(lengths):
    return _ints([0] + torch.tensor(lengths).cumsum(0).tolist())


def _normal(shape, dtype, g):
    return torch.randn(shape, device="cuda", generator=g, dtype=torch.float32).to(DTYPES[dtype])


def prepare(case, seed):
    return {"prompt": _prepare_prompt, "cached": _prepare_cached, "pages": _prepare_pages}[case["op"]](case, _generator(seed))


def _prepare_prompt(case, g):
    nq, nk = _prompt_lengths(case)
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    return dict(case=case, q=_normal((sum(nq), h, d), case["dtype"], g), k=_normal((sum(nk), kv, d), case["dtype"], g),
                v=_normal((sum(nk), kv, d), case["dtype"], g), cu_q=_starts(nq), cu_k=_starts(nk), max_q=max(nq), max_k=max(nk),
                out=torch.empty((sum(nq), h, d), dtype=DTYPES[case["dtype"]], device="cuda"),
                lse=torch.empty((sum(nq), h), dtype=torch.float32, device="cuda"))


def _tables(lengths, case, max_pages, n_pages, g):
    """Tables, lengths, pages held and reference counts of sequences whose pages lie anywhere in the pool."""
    held = [-(-n // case["page"]) for n in lengths]
    order = torch.randperm(n_pages, device="cuda", generator=g)[:sum(held)].to(torch.int32)
    table = torch.full((len(lengths), max_pages), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max_pages, device="cuda") < _ints(held)[:, None]] = order
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[order.long()] = 1
    return dict(table=table, length=_ints(lengths), held=_ints(held), refs=refs)


def _prepare_cached(case, g):
    total, draft = _cached_lengths(case)
    h, kv, d, page, n = case["heads"], case["kv_heads"], case["dim"], case["page"], case["seqs"]
    n_pages = sum(-(-t // page) for t in total) + 7
    max_pages = -(-max(total) // page) + 3
    # each drafted token's parent is an earlier one of its tree, or none (a root)
    parents = [max(j - 1 - (j * 5 + i) % 3, -1) for i, m in enumerate(draft) for j in range(m)]
    s = dict(case=case, pages=_normal((2, n_pages, page, kv, d), case["dtype"], g), seqs=_ints(list(range(n))), cu_q=_starts(draft),
             q=_normal((sum(draft), h, d), case["dtype"], g), parents=_ints(parents), max_q=max(draft),
             max_k=max(total), out=torch.empty((sum(draft), h, d), dtype=DTYPES[case["dtype"]], device="cuda"),
             lse=torch.empty((sum(draft), h), dtype=torch.float32, device="cuda"),
             mask=torch.zeros((sum(draft), -(-max(draft) // 32)), dtype=torch.int32, device="cuda"))
    return s | _tables(total, case, max_pages, n_pages, g)


def _prepare_pages(case, g):
    kv, d, page, n, kind = case["kv_heads"], case["dim"], case["page"], case["seqs"], case["kind"]
    base = _lengths(case["lo"], case["hi"], n, 4)
    draft = _lengths(case["draft_lo"], case["draft_hi"], n, 5) if kind == "step" else [1] * n
    children = case["children"] if kind == "fork" else 0
    rows = base + [0] * (n * children)
    grown = [b + m for b, m in zip(base, draft)]
    max_pages = -(-max(grown) // page) + 1
    n_pages = sum(-(-t // page) for t in grown) + 2 * n * children + 5
    s = dict(case=case, pages=_normal((2 * case["layers"], n_pages, page, kv, d), case["dtype"], g), seqs=_ints(list(range(n))),
             base=_ints(base))
    # where half of the sequences will end, they lie one after the other in the pool, that half in its front
    s |= (_rows_in_order if kind == "compact" else _tables)(rows, case, max_pages, n_pages, g)
    if kind == "step":
        kept = _kept(draft)
        place = torch.arange(max(draft), device="cuda")
        order = torch.rand((n, max(draft)), device="cuda", generator=g)
        order = order.masked_fill(place >= _ints(draft)[:, None], 2.0).argsort(dim=1)
        order = order.masked_fill(place >= _ints(kept)[:, None], 1 << 19).sort(dim=1).values  # those kept, in ascending order
        s |= dict(draft=_ints(draft), cu=_starts(draft), kept=_ints(kept), keep=order.to(torch.int32),
                  k=_normal((sum(draft), kv, d), case["dtype"], g), v=_normal((sum(draft), kv, d), case["dtype"], g))
    if kind == "fork":
        s |= dict(src=s["seqs"].repeat_interleave(children), dst=_ints(list(range(n, n + n * children))),
                  one=_ints([1] * n * children), zero=_ints([0] * n * children))
    if kind == "compact":
        half = n // 2
        s |= dict(low=s["seqs"][:half], high=s["seqs"][half:], zeros=_ints([0] * n), flip=False)
    return s


def _kept(draft):
    """How many of a sequence's drafted tokens are accepted."""
    return [1 + (i * 3) % m for i, m in enumerate(draft)]


def _rows_in_order(lengths, case, max_pages, n_pages, g):
    held = [-(-n // case["page"]) for n in lengths]
    table = torch.full((len(lengths), max_pages), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max_pages, device="cuda") < _ints(held)[:, None]] = torch.arange(sum(held), dtype=torch.int32, device="cuda")
    refs = (torch.arange(n_pages, device="cuda") < sum(held)).to(torch.int32)
    return dict(table=table, length=_ints(lengths), held=_ints(held), refs=refs)


# --------------------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "cached": _own_cached, "pages": _own_pages}[op](s)
    return {"prompt": _plain_prompt, "cached": _plain_cached, "pages": _plain_pages}[op](s)


def _own_prompt(s):
    from nvfp4_block_scaled_gather_gb300 import attention as A
    A.moe_attention_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _cache(s):
    """The handle that a program keeps over its cache."""
    if "cache" not in s:
        from nvfp4_block_scaled_gather_gb300 import attention as A
        s["cache"] = A.KVCache(s["pages"], s["table"], s["length"], s["held"], s["refs"])
    return s["cache"]


def _own_cached(s):
    from nvfp4_block_scaled_gather_gb300 import attention as A
    cache, mask = _cache(s), None
    if s["max_q"] > 1:
        mask = s["mask"]
        A.moe_tree_mask(s["parents"], s["cu_q"], mask)
    if "workspace" not in s:
        s["workspace"] = A.cached_workspace(cache, s["seqs"].numel(), s["q"].shape[0], s["q"].shape[1])
    A.moe_attention_cached(s["q"], cache, 0, s["seqs"], s["cu_q"], s["out"], s["workspace"], mask=mask, lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_pages(s):
    from nvfp4_block_scaled_gather_gb300 import attention as A
    cache, kind = _cache(s), s["case"]["kind"]
    if "workspace" not in s:
        s["workspace"] = A.pages_workspace(cache)
    if kind == "step":
        A.moe_kv_truncate(cache, s["seqs"], s["base"])
        A.moe_kv_extend(cache, s["seqs"], s["draft"], s["workspace"])
        A.moe_kv_append(cache, 0, s["seqs"], s["cu"], s["k"], s["v"])
        A.moe_kv_keep(cache, s["seqs"], s["draft"], s["keep"], s["kept"], s["workspace"])
    elif kind == "fork":
        A.moe_kv_truncate(cache, s["dst"], s["zero"])
        A.moe_kv_fork(cache, s["src"], s["dst"])
        A.moe_kv_extend(cache, s["dst"], s["one"], s["workspace"])
    else:
        gone = s["high"] if s["flip"] else s["low"]
        s["flip"] = not s["flip"]
        A.moe_kv_truncate(cache, gone, s["zeros"][:gone.numel()])
        A.moe_kv_compact(cache, s["workspace"])
        A.moe_kv_extend(cache, gone, _base_of(s, gone), s["workspace"])
    return _cache_outputs(s)


def _base_of(s, gone):
    half = s["low"].numel()
    return s["base"][:half] if gone is s["low"] else s["base"][half:]


def _cache_outputs(s):
    return {"pages": s["pages"].view(torch.int16), "table": s["table"], "length": s["length"], "held": s["held"], "refs": s["refs"]}


# --------------------------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------------------------

def _softmax_over(q, k, v, seen):
    """q [B, n, H, D], k and v [B, m, Hkv, D], seen [B, n, m]: outputs and log-sums in 32 bits."""
    b, n, h, d = q.shape
    kv = k.shape[2]
    q = q.float().reshape(b, n, kv, h // kv, d).permute(0, 2, 3, 1, 4) * (d ** -0.5)
    k, v = k.float().permute(0, 2, 3, 1)[:, :, None], v.float().permute(0, 2, 1, 3)[:, :, None]
    x = (q.reshape(b, kv, -1, d)[:, :, None] @ k).reshape(b, kv, h // kv, n, -1)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x.reshape(b, kv, 1, -1, x.shape[-1]) @ v).reshape(b, kv, h // kv, n, d) / total.clamp_min(1e-30)
    lse = (total.log() + top)[..., 0]
    return out.permute(0, 3, 1, 2, 4).reshape(b, n, h, d), lse.permute(0, 3, 1, 2).reshape(b, n, h)


def _rows(cu, width):
    """For packed rows: where each sequence's j-th row would be, and whether it is there. [B, width] both."""
    at = cu[:-1, None].long() + torch.arange(width, device="cuda")
    there = at < cu[1:, None]
    return at, there


def _plain_prompt(s):
    iq, tq = _rows(s["cu_q"], s["max_q"])
    ik, tk = _rows(s["cu_k"], s["max_k"])
    nq, nk = s["cu_q"].diff(), s["cu_k"].diff()
    limit = torch.arange(s["max_q"], device="cuda") + (nk - nq)[:, None]
    seen = (torch.arange(s["max_k"], device="cuda") <= limit[:, :, None]) & tk[:, None]
    last = [x.shape[0] - 1 for x in (s["q"], s["k"])]
    k, v = s["k"][ik.clamp_max(last[1])], s["v"][ik.clamp_max(last[1])]
    out, lse = _softmax_over(s["q"][iq.clamp_max(last[0])], k, v, seen)
    return {"out": out[tq].to(s["out"].dtype), "lse": lse[tq]}


def _ancestors(parents, cu, width):
    """Which of its tree's tokens each drafted token sees: itself and its ancestors. [B, width, width]."""
    at, there = _rows(cu, width)
    up = parents[at.clamp_max(parents.numel() - 1)].long().masked_fill(~there, -1)
    place = torch.arange(width, device="cuda")
    step = (up[:, :, None] == place).float()
    seen = torch.matrix_power(torch.eye(width, device="cuda") + step, width)  # the ways up, of any number of steps
    return seen > 0, at, there


def _plain_cached(s):
    page = s["case"]["page"]
    seen_tree, iq, tq = _ancestors(s["parents"], s["cu_q"], s["max_q"])
    length, n = s["length"][s["seqs"].long()], s["cu_q"].diff()
    place = torch.arange(s["max_k"], device="cuda")
    rows = s["table"][s["seqs"].long()][:, place // page].clamp_min(0).long()
    k, v = s["pages"][0][rows, place % page], s["pages"][1][rows, place % page]
    context = (length - n)[:, None]
    drafted = (place - context).clamp(0, s["max_q"] - 1)[:, None].expand(-1, s["max_q"], -1)
    seen = (place < context)[:, None] | (seen_tree.gather(2, drafted) & (place >= context)[:, None])
    seen &= (place < length[:, None])[:, None]
    out, lse = _softmax_over(s["q"][iq.clamp_max(s["q"].shape[0] - 1)], k, v, seen)
    return {"out": out[tq].to(s["out"].dtype), "lse": lse[tq]}


def _truncate(s, seqs, to):
    seqs, page = seqs.long(), s["case"]["page"]
    length = torch.minimum(s["length"][seqs], to)
    keep = (length + page - 1) // page
    column = torch.arange(s["table"].shape[1], device="cuda")
    gone = (column >= keep[:, None]) & (column < s["held"][seqs][:, None])
    rows = s["table"][seqs]
    s["refs"].index_add_(0, rows.clamp_min(0).flatten().long(), -gone.flatten().to(torch.int32))
    s["table"][seqs] = rows.masked_fill(gone, -1)
    s["length"][seqs], s["held"][seqs] = length, torch.minimum(keep, s["held"][seqs])


def _extend(s, seqs, add):
    seqs, page = seqs.long(), s["case"]["page"]
    length, held, rows = s["length"][seqs], s["held"][seqs], s["table"][seqs]
    need = ((length + add + page - 1) // page - held).clamp_min(0)
    opened = (length % page != 0) & (add > 0)
    last = rows.gather(1, (length // page).clamp_max(rows.shape[1] - 1)[:, None].long())[:, 0].clamp_min(0).long()
    same = (last[:, None] == last) & opened[:, None] & opened
    copied = opened & (s["refs"][last] - same.tril(-1).sum(1) > 1)
    want = need + copied
    first = want.cumsum(0) - want
    free = (s["refs"] != 0).sort(stable=True).indices  # the free pages, lowest first
    j = torch.arange(rows.shape[1] + 1, device="cuda")
    taken = j < want[:, None]
    fresh = free[(first[:, None] + j).clamp_max(free.numel() - 1)]
    column = torch.where((j == 0) & copied[:, None], (length // page)[:, None], held[:, None] + j - copied[:, None].int())
    s["table"][seqs[:, None].expand_as(column)[taken], column[taken]] = fresh[taken].to(torch.int32)
    s["refs"].index_add_(0, last, -copied.to(torch.int32))
    s["refs"][fresh[taken]] = 1
    src, dst = last[copied], fresh[:, 0][copied]
    used = (torch.arange(page, device="cuda") < (length % page)[copied][:, None])[None, :, :, None, None]
    s["pages"][:, dst] = torch.where(used, s["pages"][:, src], s["pages"][:, dst])
    s["length"][seqs], s["held"][seqs] = length + add, held + need


def _places(s, seqs, at):
    """The page and the row in it of the tokens at the places `at` [n, m] of the sequences."""
    page = s["case"]["page"]
    return s["table"][seqs.long()].gather(1, (at // page).clamp(0, s["table"].shape[1] - 1).long()).long(), (at % page).long()


def _append(s, seqs, cu, k, v):
    i, there = _rows(cu, s["keep"].shape[1])
    at = (s["length"][seqs.long()] - cu.diff())[:, None] + torch.arange(i.shape[1], device="cuda")
    page, row = _places(s, seqs, at)
    s["pages"][0][page[there], row[there]] = k[i[there]]
    s["pages"][1][page[there], row[there]] = v[i[there]]


def _keep(s, seqs, draft, keep, kept):
    start = (s["length"][seqs.long()] - draft)[:, None]
    j = torch.arange(keep.shape[1], device="cuda")
    there = j < kept[:, None]
    sp, sr = _places(s, seqs, start + keep)
    dp, dr = _places(s, seqs, start + j)
    s["pages"][:, dp[there], dr[there]] = s["pages"][:, sp[there], sr[there]]
    _truncate(s, seqs, start[:, 0] + kept)


def _fork(s, src, dst):
    src, dst = src.long(), dst.long()
    rows = s["table"][src]
    s["table"][dst], s["length"][dst], s["held"][dst] = rows, s["length"][src], s["held"][src]
    s["refs"].index_add_(0, rows.clamp_min(0).flatten().long(), (rows >= 0).flatten().to(torch.int32))


def _compact(s):
    used = s["refs"] > 0
    place = torch.arange(used.numel(), device="cuda")
    count = used.sum()
    src, dst = place[used & (place >= count)], place[~used & (place < count)]
    moved = place.clone()
    moved[src] = dst
    s["pages"][:, dst] = s["pages"][:, src]
    s["table"].copy_(torch.where(s["table"] >= 0, moved[s["table"].clamp_min(0).long()].to(torch.int32), s["table"]))
    s["refs"][dst], s["refs"][src] = s["refs"][src], 0


def _plain_pages(s):
    kind = s["case"]["kind"]
    if kind == "step":
        _truncate(s, s["seqs"], s["base"])
        _extend(s, s["seqs"], s["draft"])
        _append(s, s["seqs"], s["cu"], s["k"], s["v"])
        _keep(s, s["seqs"], s["draft"], s["keep"], s["kept"])
    elif kind == "fork":
        _truncate(s, s["dst"], s["zero"])
        _fork(s, s["src"], s["dst"])
        _extend(s, s["dst"], s["one"])
    else:
        gone = s["high"] if s["flip"] else s["low"]
        s["flip"] = not s["flip"]
        _truncate(s, gone, s["zeros"][:gone.numel()])
        _compact(s)
        _extend(s, gone, _base_of(s, gone))
    return _cache_outputs(s)


# --------------------------------------------------------------------------------------------------------------
# the definition in 64 bits, and the work
# --------------------------------------------------------------------------------------------------------------

def _one_exact(q, k, v, seen):
    """q [n, H, D], k and v [m, Hkv, D], seen [n, m], one sequence."""
    n, h, d = q.shape
    out = torch.zeros((n, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((n, h), -math.inf, dtype=torch.float64, device="cuda")
    some = seen.any(1)
    for head in range(h):
        kv = head // (h // k.shape[1])
        x = torch.einsum("nd,md->nm", q[:, head].double(), k[:, kv].double()) / math.sqrt(d)
        x = torch.where(seen, x, torch.full_like(x, -math.inf))[some]
        lse[some, head] = torch.logsumexp(x, 1)
        out[some, head] = torch.exp(x - lse[some, head][:, None]) @ v[:, kv].double()
    return out, lse


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers and moved bits: nothing is computed
    s = prepare(case, seed)
    outs, lses, cu = [], [], s["cu_q"].tolist()
    for b in range(case["seqs"]):
        q = s["q"][cu[b]:cu[b + 1]]
        n = q.shape[0]
        if case["op"] == "prompt":
            lo, hi = s["cu_k"][b].item(), s["cu_k"][b + 1].item()
            k, v = s["k"][lo:hi], s["v"][lo:hi]
            seen = torch.ones((n, hi - lo), device="cuda").tril(hi - lo - n) > 0
        else:
            m, page = s["length"][b].item(), case["page"]
            pages = s["table"][b, :-(-m // page)].long()
            k, v = (s["pages"][i][pages].flatten(0, 1)[:m] for i in (0, 1))
            seen = torch.zeros((n, m), dtype=torch.bool)
            seen[:, :m - n] = True
            parents = s["parents"][cu[b]:cu[b + 1]].tolist()
            for i in range(n):
                j = i
                while j >= 0:
                    seen[i, m - n + j] = True
                    j = parents[j]
            seen = seen.cuda()
        o, e = _one_exact(q, k, v, seen)
        outs.append(o)
        lses.append(e)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def work(case):
    if case["op"] == "pages":
        return _pages_work(case)
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "prompt":
        nq, nk = _prompt_lengths(case)
        pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(nq, nk))
    else:
        nk, nq = _cached_lengths(case)
        pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(nq, nk))
    return {"bytes": 2 * sum(nk) * kv * d * 2 + sum(nq) * h * (4 * d + 4), "flops": 4 * d * h * pairs}


def _pages_work(case):
    row, n = case["kv_heads"] * case["dim"] * 2, case["seqs"]
    planes, page = 2 * case["layers"], case["page"]
    base = _lengths(case["lo"], case["hi"], n, 4)
    tables = 4 * sum(-(-b // page) for b in base)
    if case["kind"] == "step":
        draft = _lengths(case["draft_lo"], case["draft_hi"], n, 5)
        kept = _kept(draft)
        return {"bytes": 4 * sum(draft) * row + 2 * planes * row * sum(kept) + tables, "flops": 0}
    if case["kind"] == "fork":
        return {"bytes": 2 * planes * row * case["children"] * sum(b % page for b in base) + 2 * case["children"] * tables, "flops": 0}
    half = [-(-b // page) for b in base]
    return {"bytes": 2 * planes * row * page * min(sum(half[:n // 2]), sum(half[n // 2:])) + 2 * tables, "flops": 0}
