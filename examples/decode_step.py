#!/usr/bin/env python3
"""Speculative decode steps over a paged cache, with every operator of the
library where a serving loop has it.

With --prompt N each request starts from a prompt of its own length: its keys
and values go into the cache and prompt_attention answers all prompts, packed
one behind another, in one call.  With --four-bit the cache holds 4 bits an
element.  Either has norms and rotated positions.

Each step of a small random model with one attention layer:
  1. the queries, keys and values of each request's draft tree (its last token
     and the drafts below it) go into the cache (rotate_and_cache);
  2. an indexer's scores select the cache entries of the last token
     (top_k_page_table_transform) and selected_attention reads those alone;
     tree_attention reads the whole cache for all nodes of the tree;
  3. verify_drafts decides which drafts stand and draws the next token;
  4. accumulate_cache_weights adds what the accepted nodes paid attention to;
  5. evict_cache drops the refused drafts, and the positions of least weight
     once a request is over its budget, into fresh pages (the old ones free).

    python examples/decode_step.py [--steps 12] [--batch 4] [--prompt 0] [--four-bit]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_top_gb300 as gb  # noqa: E402

NODES, PAGE, BUDGET, RECENT, WIDTH = 8, 16, 48, 16, 128
Q_HEADS, KV_HEADS, DIM, VOCAB = 8, 2, 64, 997
# parents of the tree's nodes: a chain of four and two side branches
PARENTS = [0, 0, 1, 2, 0, 4, 1, 6]


def tree_bits(batch, device):
    rows = []
    for n in range(NODES):
        rows.append((rows[PARENTS[n]] if n else 0) | 1 << n)
    return torch.tensor(rows * batch, dtype=torch.int64, device=device)


class Model:
    """Random projections: embedding -> attention -> logits."""

    def __init__(self, device, g):
        def w(*shape):
            return (torch.randn(shape, generator=g, device=device) / shape[0] ** 0.5).to(torch.bfloat16)
        self.embed = torch.randn((VOCAB, 128), generator=g, device=device).to(torch.bfloat16)
        self.q, self.k, self.v = w(128, Q_HEADS * DIM), w(128, KV_HEADS * DIM), w(128, KV_HEADS * DIM)
        self.out = w(Q_HEADS * DIM, VOCAB)


class Cache:
    """A paged cache of 16 or 4 bits an element, by the calls that differ."""

    def __init__(self, slots, four_bit, device):
        self.four_bit = four_bit
        if four_bit:
            self.rows = torch.zeros((slots, KV_HEADS, gb.int4_row_bytes(DIM)), dtype=torch.uint8, device=device)
            self.parts = gb.int4_parts(self.rows)
            self.all = torch.arange(slots, dtype=torch.int32, device=device)
        else:
            self.parts = torch.zeros((2, slots, KV_HEADS, DIM), dtype=torch.bfloat16, device=device).unbind(0)

    def write(self, q, k, v, positions, slots, **kw):
        if self.four_bit:
            return gb.rotate_and_cache_int4(q, k, v, positions, slots, kw.pop("freqs"), self.rows, **kw)
        return gb.rotate_and_cache(q, k, v, positions, slots, kw.pop("freqs"), *self.parts, **kw)

    def tree_attention(self, q, *args, **kw):
        return gb.tree_attention_int4(q, self.rows, *args, **kw) if self.four_bit else gb.tree_attention(q, *self.parts, *args, **kw)

    def selected_attention(self, q, chosen):
        return gb.selected_attention_int4(q, self.rows, chosen) if self.four_bit else gb.selected_attention(q, *self.parts, chosen)

    def keys(self):
        return gb.read_cache_int4(self.rows, self.all, DIM).k if self.four_bit else self.parts[0]


def run(steps=12, batch=4, device="cuda", seed=0, say=print, prompt=0, four_bit=False):
    """Runs the loop; returns the tokens of each request."""
    dev = torch.device(device)
    g = torch.Generator(device=dev).manual_seed(seed)
    model, tree = Model(dev, g), tree_bits(batch, dev)
    cols = WIDTH // PAGE
    # two sets of pages a request: a step reads one and packs into the other
    pages = torch.randperm(2 * batch * cols, generator=g, device=dev).to(torch.int32).view(2, batch, cols)
    cache = Cache(2 * batch * cols * PAGE, four_bit, dev)
    weights = torch.zeros((batch, KV_HEADS, WIDTH), device=dev)
    lens = torch.zeros(batch, dtype=torch.int32, device=dev)       # positions that stand
    last = torch.randint(0, VOCAB, (batch,), generator=g, device=dev, dtype=torch.int32)
    node = torch.arange(NODES, device=dev)
    turned = prompt > 0 or four_bit
    freqs = 1e4 ** (-torch.arange(DIM // 2, device=dev) / (DIM // 2)) if turned else None
    norm = torch.ones(DIM, device=dev) if turned else None
    how = dict(freqs=freqs, q_weight=norm, k_weight=norm)
    depth = torch.tensor([bin(int(x) & (1 << NODES) - 1).count("1") - 1 for x in tree[:NODES]], device=dev)
    said = [[int(t)] for t in last]
    seen = torch.zeros(batch, dtype=torch.int32, device=dev)       # tokens so far: their places turn the heads

    def slots_of(table, rows, pos):
        return (table[rows, (pos // PAGE).long()] * PAGE + pos % PAGE).to(torch.int32)

    def heads(x):
        return (x @ model.q).view(-1, Q_HEADS, DIM), (x @ model.k).view(-1, KV_HEADS, DIM), (x @ model.v).view(-1, KV_HEADS, DIM)

    if prompt:
        each = torch.randint(max(1, prompt // 2), prompt + 1, (batch,), generator=g, device=dev)
        cu = torch.nn.functional.pad(each.cumsum(0), (1, 0)).to(torch.int32)
        rows = torch.repeat_interleave(torch.arange(batch, device=dev), each)
        pos = (torch.arange(rows.numel(), device=dev) - cu[rows]).to(torch.int32)
        words = torch.randint(0, VOCAB, (rows.numel(),), generator=g, device=dev)
        q, k, v = heads(model.embed[words])
        q = cache.write(q, k, v, pos, slots_of(pages[0], rows, pos), **how)
        # the keys as they were cached, for the prompts' own attention
        at = slots_of(pages[0], rows, pos)
        k, v = gb.read_cache_int4(cache.rows, at, DIM) if four_bit else (x[at.long()] for x in cache.parts)
        att = gb.prompt_attention(q, k, v, cu)
        first = (att[(cu[1:] - 1).long()].view(batch, -1) @ model.out).float().argmax(1)
        lens, seen, last = each.to(torch.int32), each.to(torch.int32), first.to(torch.int32)
        said = [[int(t)] for t in last]
    for step in range(steps):
        # the drafts: here the words that a noisy copy of the model would say
        tokens = torch.randint(0, VOCAB, (batch, NODES), generator=g, device=dev, dtype=torch.int32)
        tokens[:, 0] = last
        x = model.embed[tokens.long()].view(batch * NODES, 128)
        seq = lens + NODES
        pos = lens.unsqueeze(1) + node
        table = pages[step % 2]
        at = table.gather(1, (pos // PAGE).long()) * PAGE + (pos % PAGE).to(torch.int32)
        q, k, v = heads(x)
        q = cache.write(q, k, v, (seen.unsqueeze(1) + depth).to(torch.int32).view(-1), at.to(torch.int32).view(-1), **how)

        att, lse = cache.tree_attention(q, table, seq, page_size=PAGE, next_n=NODES, tree_mask=tree, return_lse=True)
        # the last token once more over an indexer's selection of its context
        root = q.view(batch, NODES, Q_HEADS, DIM)[:, 0].contiguous()
        scores = torch.randn((batch, WIDTH), generator=g, device=dev)
        chosen = gb.top_k_page_table_transform(scores, lens + 1, table, 64, page_size=PAGE)
        sparse = cache.selected_attention(root, chosen)
        att = att.view(batch, NODES, -1)
        att[:, 0] = 0.5 * (att[:, 0] + sparse.view(batch, -1))

        logits = (att.view(batch * NODES, -1) @ model.out).float() * 40
        # half of the drafts are the target's own first words, so that some stand
        likely = logits.view(batch, NODES, VOCAB).argmax(2).to(torch.int32)
        guess = likely.gather(1, torch.tensor(PARENTS, device=dev).expand(batch, NODES))
        tokens = torch.where((node > 0) & (torch.rand((batch, NODES), generator=g, device=dev) < 0.5), guess, tokens)
        got = gb.verify_drafts(logits, tokens.view(-1).contiguous(), torch.rand(batch * NODES, generator=g, device=dev),
                               torch.empty((batch, VOCAB), device=dev).exponential_(generator=g).clamp_(min=1e-20),
                               next_n=NODES, tree_mask=tree)
        gb.accumulate_cache_weights(q, cache.keys(), lse, table, seq, weights, page_size=PAGE, next_n=NODES, tree_mask=tree,
                                    accept_mask=got.accept_mask)
        kept = gb.evict_cache(weights, *cache.parts, table, seq, pages[(step + 1) % 2], BUDGET, recent=RECENT,
                              page_size=PAGE, next_n=NODES, accept_mask=got.accept_mask)
        weights, lens, last = kept.weights, kept.new_lens, got.next_token
        seen = seen + got.accepted + 1
        for i in range(batch):
            said[i] += [int(tokens[i, n]) for n in got.path[i, 1:].tolist() if n >= 0] + [int(last[i])]
        say(f"step {step}: accepted {got.accepted.tolist()}, cached {lens.tolist()}")
    return said


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=0, help=f"tokens of the longest prompt, at most {WIDTH - NODES}")
    ap.add_argument("--four-bit", action="store_true")
    a = ap.parse_args()
    for i, words in enumerate(run(a.steps, a.batch, prompt=a.prompt, four_bit=a.four_bit)):
        print(f"request {i}: {len(words)} tokens, the last {words[-8:]}")


if __name__ == "__main__":
    main()
