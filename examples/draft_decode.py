"""Serving with drafted trees, every operator in its place: a small decoder of
random weights whose blocks are attention over the paged cache and the
routed-expert NVFP4 layer.

  prompts    moe_kv_extend, then in each block moe_kv_append,
             moe_attention_prompt and moe_nvfp4_layer
  drafting   moe_kv_fork: a copy of each sequence that shares its pages decodes
             one token at a time (moe_attention_cached) and so finds what the
             model would say; moe_kv_truncate lets go of it
  verifying  the drafted tokens with wrong siblings form a tree: moe_tree_mask,
             moe_attention_cached with the mask, and moe_kv_keep of the path
             that the model agrees with
  upkeep     a sequence ends (moe_kv_truncate) and moe_kv_compact moves the
             pages in use to the front

Run: python examples/draft_decode.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_block_scaled_gather_gb300 import _native as N  # noqa: E402
from nvfp4_block_scaled_gather_gb300 import attention as A  # noqa: E402
from nvfp4_block_scaled_gather_gb300.synthetic import CONFIGS, make_weights  # noqa: E402

LAYERS, HEADS, KV_HEADS, DIM, VOCAB = 2, 8, 2, 64, 512
PAGE, MAX_TOKENS, MAX_SEQS = 16, 512, 16
CFG = CONFIGS["tiny"]


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def starts(counts):
    return ints([sum(counts[:i]) for i in range(len(counts) + 1)])


def norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Decoder:
    """Blocks of attention and routed experts; attend(layer, q, k, v) is the caller's."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def draw(rows, columns):
            return torch.randn((rows, columns), device="cuda", generator=g).mul_(rows ** -0.5).bfloat16()

        h = CFG.H
        self.embed = torch.randn((VOCAB, h), device="cuda", generator=g).bfloat16()
        self.head = draw(h, VOCAB)
        self.qkv = [draw(h, (HEADS + 2 * KV_HEADS) * DIM) for _ in range(LAYERS)]
        self.out = [draw(HEADS * DIM, h) for _ in range(LAYERS)]
        self.router = [draw(h, CFG.E) for _ in range(LAYERS)]
        self.experts = []
        for layer in range(LAYERS):
            w = make_weights(CFG.E, h, CFG.I, seed=layer, device="cuda")
            w = N.Weights(*(w[k] for k in ("w13_packed", "w13_sf_linear", "g_gate_up", "w2_packed", "w2_sf_linear",
                                           "g_down")))
            self.experts.append(N.MoeLayer(w, MAX_TOKENS, CFG.k))

    def __call__(self, tokens, attend):
        """The token that the model says after each of `tokens`."""
        h = self.embed[tokens.long()]
        for layer in range(LAYERS):
            # q, k and v are views of one product's rows: their strides go along
            x = (norm(h) @ self.qkv[layer]).view(-1, HEADS + 2 * KV_HEADS, DIM)
            a = attend(layer, x[:, :HEADS], x[:, HEADS:HEADS + KV_HEADS], x[:, HEADS + KV_HEADS:])
            h = h + a.reshape(-1, HEADS * DIM) @ self.out[layer]
            x = norm(h)
            weight, ids = torch.topk(torch.softmax((x @ self.router[layer]).float(), -1), CFG.k)
            h = h + norm(self.experts[layer](x, ids.int().contiguous(), weight.contiguous()))
        return (norm(h) @ self.head).argmax(-1).int()


class Server:
    def __init__(self, seed=0):
        self.model = Decoder(seed)
        pages = MAX_SEQS * MAX_TOKENS // PAGE
        self.cache = A.KVCache.empty(LAYERS, pages, PAGE, KV_HEADS, DIM, MAX_SEQS, MAX_TOKENS // PAGE)
        self.pages_ws = A.pages_workspace(self.cache)
        self.attn_ws = A.cached_workspace(self.cache, MAX_SEQS, MAX_TOKENS, HEADS)

    def step(self, seqs, tokens, prompt=False, parents=None):
        """Puts each sequence's tokens (a list each) into the cache and returns
        what the model says after every one of them, as lists."""
        counts = [len(t) for t in tokens]
        ids, cu = ints(seqs), starts(counts)
        A.moe_kv_extend(self.cache, ids, ints(counts), self.pages_ws)
        mask = None
        if parents is not None:
            mask = torch.empty((sum(counts), (max(counts) + 31) // 32), dtype=torch.int32, device="cuda")
            A.moe_tree_mask(ints(sum(parents, [])), cu, mask)

        def attend(layer, q, k, v):
            out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
            A.moe_kv_append(self.cache, layer, ids, cu, k, v)
            if prompt:
                A.moe_attention_prompt(q, k, v, cu, cu, out)
            else:
                A.moe_attention_cached(q, self.cache, layer, ids, cu, out, self.attn_ws, mask=mask)
            return out

        says = self.model(ints(sum(tokens, [])), attend).tolist()
        return [says[sum(counts[:i]):sum(counts[:i + 1])] for i in range(len(counts))]

    def draft(self, seqs, following, steps):
        """What the model would say after each sequence's next token, by copies that share the sequences' pages."""
        copies = list(range(MAX_SEQS - len(seqs), MAX_SEQS))
        A.moe_kv_fork(self.cache, ints(seqs), ints(copies))
        lines = [[t] for t in following]
        for _ in range(steps):
            says = self.step(copies, [[line[-1]] for line in lines])
            lines = [line + s[-1:] for line, s in zip(lines, says)]
        A.moe_kv_truncate(self.cache, ints(copies), ints([0] * len(copies)))
        return lines

    def verify(self, seqs, lines):
        """One step over a tree a sequence: its line, each token of it with a
        wrong sibling. Keeps what the model agrees with; returns the accepted
        tokens and the one after them of each sequence."""
        tokens, parents = [], []
        for line in lines:
            t, p, last = [line[0]], [-1], 0
            for x in line[1:]:
                t += [(x + 1) % VOCAB, x]
                p += [last, last]
                last = len(t) - 1
            tokens.append(t)
            parents.append(p)
        says = self.step(seqs, tokens, parents=parents)
        keep, results = [], []
        for t, p, s in zip(tokens, parents, says):
            path = [0]  # the first token is the model's own
            while True:
                agreed = [c for c in range(len(t)) if p[c] == path[-1] and t[c] == s[path[-1]]]
                if not agreed:
                    break
                path.append(agreed[0])
            keep.append(path)
            results.append(([t[c] for c in path], s[path[-1]]))
        width = max(map(len, keep))
        A.moe_kv_keep(self.cache, ints(seqs), ints([len(t) for t in tokens]),
                      ints([k + [0] * (width - len(k)) for k in keep]), ints([len(k) for k in keep]), self.pages_ws)
        return results

    def end(self, seqs):
        A.moe_kv_truncate(self.cache, ints(seqs), ints([0] * len(seqs)))
        A.moe_kv_compact(self.cache, self.pages_ws)


def run(prompts=(37, 5, 130), drafted=6, rounds=4, seed=0):
    """(the server, each live sequence's tokens, tokens accepted per verifying step)"""
    g = torch.Generator().manual_seed(seed)
    server = Server(seed)
    history = [torch.randint(0, VOCAB, (n,), generator=g).tolist() for n in prompts]
    seqs = list(range(len(prompts)))
    following = [s[-1] for s in server.step(seqs, history, prompt=True)]
    accepted = []
    for r in range(rounds):
        results = server.verify(seqs, server.draft(seqs, following, drafted))
        for i, (kept, _) in zip(seqs, results):
            history[i] += kept
            accepted.append(len(kept))
        following = [nxt for _, nxt in results]
        if r == rounds // 2:  # the first sequence ends
            server.end(seqs[:1])
            seqs, following = seqs[1:], following[1:]
    torch.cuda.synchronize()
    status = N.check_status()
    if status:
        raise RuntimeError(f"device status {status}")
    return server, {i: history[i] for i in seqs}, accepted


if __name__ == "__main__":
    server, live, accepted = run()
    print(f"{len(accepted)} verifying steps kept {sum(accepted)} tokens; "
          f"live sequences hold {[len(t) for t in live.values()]} tokens in "
          f"{int((server.cache.refs > 0).sum())} pages")
