"""A model in front of the constrained decode step, with branches of the catalog
drafted and verified in one forward pass.

Four sequences share a prompt: it is read once, causally, into the paged cache
and forked (its pages are shared until they are written).  Then each round

  1. drafts, for every sequence, the branches of the catalog's trie below the
     token it emitted last (PagePool.reserve makes room, and says which shared
     page has to be copied first: KvCache.copy_pages);
  2. runs the model over the drafts: per layer KvCache.append (norms of queries
     and keys, rotation, write into the cache) and KvCache.attend under the
     trees' masks (tree_masks);
  3. takes constrained steps (Context.step) along the branches, as long as every
     sequence's emitted token was drafted;
  4. moves the accepted branches together (KvCache.compact) and gives the pages
     behind them back (PagePool.trim).

Without drafts a round is the plain decode of one token.  Weights are random;
the catalog is the 42-name one of the package's workloads.

    python examples/tree_decode.py
"""
from __future__ import annotations

import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

PAGE, PAGES, WIDTH = 16, 256, 16
Q_HEADS, KV_HEADS, HEAD_DIM, LAYERS = 8, 2, 64, 2


class Model:
    """A small pre-norm attention model (no feed-forward layers) over a tied embedding."""

    def __init__(self, tcd, emb, seed: int = 7):
        import torch
        self.tcd, self.emb, self.torch = tcd, emb, torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        hidden = emb.shape[1]

        def weights(rows, cols):
            return (torch.randn((rows, cols), generator=g, device="cuda") * rows ** -0.5).bfloat16()

        self.qkv = [weights(hidden, (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM) for _ in range(LAYERS)]
        self.out = [weights(Q_HEADS * HEAD_DIM, hidden) for _ in range(LAYERS)]
        self.norm = torch.ones(HEAD_DIM, dtype=torch.bfloat16, device="cuda")
        pool = torch.zeros((LAYERS, PAGES, 2, KV_HEADS, PAGE, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        self.cache = tcd.KvCache(pool)
        angle = torch.arange(PAGE * WIDTH, device="cuda")[:, None] * 1e4 ** (
            -torch.arange(0, HEAD_DIM, 2, device="cuda") / HEAD_DIM)
        self.rope = torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()

    def forward(self, tokens, cu, ctx, table, max_tokens, tree=None, positions=None):
        """Hidden states [tokens, hidden] of packed tokens behind `ctx` cached ones."""
        torch = self.torch
        x = self.emb[tokens].float() * 4
        for layer in range(LAYERS):
            y = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).bfloat16()
            qkv = y @ self.qkv[layer]
            q = torch.empty((len(tokens), Q_HEADS, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
            o = torch.empty_like(q)
            self.cache.append(layer, qkv, cu, ctx, table, q, q_weight=self.norm, k_weight=self.norm, rope=self.rope,
                              positions=positions)
            self.cache.attend(layer, q, cu, ctx, table, o, max_tokens, tree=tree)
            x = x + (o.flatten(1) @ self.out[layer]).float()
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Catalog:
    """The compiled trie's edges on the host, for drafting."""

    def __init__(self, trie, sep_id: int):
        e = trie.export()
        self.begin, self.tok, self.child, self.sep = e["node_begin"], e["edge_tok"], e["edge_child"], sep_id

    def edges(self, node: int):
        """(token, node after it) of a node's edges but stop; the separator leads back to the root."""
        lo, hi = self.begin[node], self.begin[node + 1]
        return [(int(t), max(int(c), 0)) for t, c in zip(self.tok[lo:hi], self.child[lo:hi]) if c != -2]

    def after(self, node: int, token: int):
        return next((c for t, c in self.edges(node) if t == token), None)

    def draft(self, token: int, node: int, size: int):
        """The emitted token and up to size - 1 continuations, level by level: tokens, parents, trie nodes."""
        toks, parents, nodes = [token], [-1], [node]
        i = 0
        while i < len(toks) and len(toks) < size:
            for t, c in self.edges(nodes[i])[:size - len(toks)]:
                toks.append(t)
                parents.append(i)
                nodes.append(c)
            i += 1
        return toks, parents, nodes


def decode(tcd, draft: int, batch: int = 4, prompt_len: int = 37, k: int = 3):
    """Decode `batch` sequences with drafts of `draft` tokens (1: none): their tokens, and the rounds taken."""
    import torch

    from trie_constrained_decoding_gb300 import inputs as I
    w = I.tiny()
    emb = torch.from_numpy(w.embedding().view(np.int16)).cuda().view(torch.bfloat16)
    ctx = tcd.Context(emb, max_batch=batch)
    trie = tcd.Trie.compile(w.catalog, w.sep_id, w.stop_id, w.vocab)
    ctx.bind(trie)
    ctx.reset(batch, k)
    catalog, model, pages = Catalog(trie, w.sep_id), Model(tcd, emb), tcd.PagePool(PAGES, PAGE)
    rng = np.random.default_rng(11)

    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    def table():
        return ints(np.stack([pages.row(s, WIDTH) for s in seqs]))

    def reserve(start, count):
        """Room for each sequence's next tokens; shared pages are copied before they are written."""
        copies = [c for s, a, n in zip(seqs, start, count) for c in pages.reserve(s, a, a + n)]
        if copies:
            model.cache.copy_pages(ints([a for a, _ in copies]), ints([b for _, b in copies]))

    # the shared prompt, read once and forked; each sequence then gets a last prompt token of its own
    shared = pages.open()
    seqs = [shared]
    pages.reserve(shared, 0, prompt_len)
    prompt = torch.from_numpy(rng.integers(0, w.vocab, prompt_len)).cuda()
    model.forward(prompt, ints([0, prompt_len]), ints([0]), table(), prompt_len)
    seqs = [shared] + [pages.fork(shared, prompt_len) for _ in range(batch - 1)]
    lens = [prompt_len] * batch
    pending = [int(t) for t in rng.integers(0, w.vocab, batch)]   # emitted (or given), not cached yet
    node = [0] * batch                                            # the trie's node after it
    toks, done, rounds = [[] for _ in range(batch)], [False] * batch, 0
    tok, logit = ints([0] * batch), torch.zeros(batch, device="cuda")
    while not all(done):
        rounds += 1
        drafts = [([], [], []) if d else catalog.draft(t, n, draft) for d, t, n in zip(done, pending, node)]
        count = [len(d[0]) for d in drafts]
        reserve(lens, count)
        cu, lens_dev, rows = ints(np.concatenate(([0], np.cumsum(count)))), ints(lens), table()
        flat = torch.tensor([t for d in drafts for t in d[0]], device="cuda")
        masks = torch.zeros((len(flat), 1), dtype=torch.int64, device="cuda")
        positions = ints([0] * len(flat))
        bad = tcd.tree_masks(ints([p for d in drafts for p in d[1]]), cu, lens_dev, masks, positions)
        hidden = model.forward(flat, cu, lens_dev, rows, max(count), masks, positions)
        model.cache.raise_on_error()    # (of every call since the last look: all layers, page copies, the prompt)
        assert not bool(bad.any())
        # constrained steps along the drafts, while every sequence's next token is one of them
        first = np.concatenate(([0], np.cumsum(count)))
        at, paths = [0] * batch, [[] if d else [0] for d in done]
        while True:
            row = torch.stack([hidden[first[b] + at[b]] if count[b] else torch.zeros_like(hidden[0])
                               for b in range(batch)])
            ctx.step(row, tok, logit)
            emitted, on = tok.tolist(), True
            for b in range(batch):
                if done[b]:
                    continue
                t = emitted[b]
                toks[b].append(t)
                if t == w.stop_id:
                    done[b] = True
                    continue
                node[b], pending[b] = catalog.after(node[b], t), t
                child = next((i for i in range(count[b]) if drafts[b][1][i] == at[b] and drafts[b][0][i] == t), None)
                if child is None:
                    on = False
                else:
                    at[b] = child
            if not on or all(done):
                break
            for b in range(batch):
                if not done[b]:
                    paths[b].append(at[b])
        ctx.raise_on_error()
        # the accepted branches move together; what lies behind them is free again
        wide = max(max(len(p) for p in paths), 1)
        after = torch.zeros_like(lens_dev)
        model.cache.compact(rows, lens_dev, ints([p + [-1] * (wide - len(p)) for p in paths]),
                            ints([len(p) for p in paths]), after)
        model.cache.raise_on_error()
        lens = after.tolist()
        for s, n in zip(seqs, lens):
            pages.trim(s, n)
    for s in seqs:
        pages.close_seq(s)
    assert pages.free == PAGES
    ctx.close()
    return toks, rounds


def main():
    from trie_constrained_decoding_gb300 import binding as tcd
    plain, steps = decode(tcd, 1)
    drafted, rounds = decode(tcd, 16)
    for b, t in enumerate(drafted):
        print(f"sequence {b}: {t}")
    print(f"plain decode: {steps} forward passes; drafts of up to 16 tokens: {rounds}; "
          f"tokens {'equal' if plain == drafted else 'differ'}")


if __name__ == "__main__":
    main()
