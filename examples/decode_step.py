#!/usr/bin/env python3
"""Speculative decode steps over a paged cache, with every operator of the
library where a serving loop has it.

Each step of a small random model with one attention layer:
  1. the queries, keys and values of each request's draft tree (its last token
     and the drafts below it) go into the cache;
  2. an indexer's scores select the cache entries of the last token
     (top_k_page_table_transform) and selected_attention reads those alone;
     tree_attention reads the whole cache for all nodes of the tree;
  3. verify_drafts decides which drafts stand and draws the next token;
  4. accumulate_cache_weights adds what the accepted nodes paid attention to;
  5. evict_cache drops the refused drafts, and the positions of least weight
     once a request is over its budget, into fresh pages (the old ones free).

    python examples/decode_step.py [--steps 12] [--batch 4]
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


def run(steps=12, batch=4, device="cuda", seed=0, say=print):
    """Runs the loop; returns the tokens of each request."""
    dev = torch.device(device)
    g = torch.Generator(device=dev).manual_seed(seed)
    model, tree = Model(dev, g), tree_bits(batch, dev)
    cols = WIDTH // PAGE
    # two sets of pages a request: a step reads one and packs into the other
    pages = torch.randperm(2 * batch * cols, generator=g, device=dev).to(torch.int32).view(2, batch, cols)
    slots = 2 * batch * cols * PAGE
    k_cache = torch.zeros((slots, KV_HEADS, DIM), dtype=torch.bfloat16, device=dev)
    v_cache = torch.zeros_like(k_cache)
    weights = torch.zeros((batch, KV_HEADS, WIDTH), device=dev)
    lens = torch.zeros(batch, dtype=torch.int32, device=dev)       # positions that stand
    last = torch.randint(0, VOCAB, (batch,), generator=g, device=dev, dtype=torch.int32)
    node = torch.arange(NODES, device=dev)
    said = [[int(t)] for t in last]
    for step in range(steps):
        # the drafts: here the words that a noisy copy of the model would say
        tokens = torch.randint(0, VOCAB, (batch, NODES), generator=g, device=dev, dtype=torch.int32)
        tokens[:, 0] = last
        x = model.embed[tokens.long()].view(batch * NODES, 128)
        q = (x @ model.q).view(-1, Q_HEADS, DIM)
        seq = lens + NODES
        pos = lens.unsqueeze(1) + node
        table = pages[step % 2]
        at = table.gather(1, (pos // PAGE).long()).long() * PAGE + pos % PAGE
        k_cache[at.view(-1)] = (x @ model.k).view(-1, KV_HEADS, DIM)
        v_cache[at.view(-1)] = (x @ model.v).view(-1, KV_HEADS, DIM)

        att, lse = gb.tree_attention(q, k_cache, v_cache, table, seq, page_size=PAGE, next_n=NODES, tree_mask=tree,
                                     return_lse=True)
        # the last token once more over an indexer's selection of its context
        root = q.view(batch, NODES, Q_HEADS, DIM)[:, 0].contiguous()
        scores = torch.randn((batch, WIDTH), generator=g, device=dev)
        chosen = gb.top_k_page_table_transform(scores, lens + 1, table, 64, page_size=PAGE)
        sparse = gb.selected_attention(root, k_cache, v_cache, chosen)
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
        gb.accumulate_cache_weights(q, k_cache, lse, table, seq, weights, page_size=PAGE, next_n=NODES, tree_mask=tree,
                                    accept_mask=got.accept_mask)
        kept = gb.evict_cache(weights, k_cache, v_cache, table, seq, pages[(step + 1) % 2], BUDGET, recent=RECENT,
                              page_size=PAGE, next_n=NODES, accept_mask=got.accept_mask)
        weights, lens, last = kept.weights, kept.new_lens, got.next_token
        for i in range(batch):
            said[i] += [int(tokens[i, n]) for n in got.path[i, 1:].tolist() if n >= 0] + [int(last[i])]
        say(f"step {step}: accepted {got.accepted.tolist()}, cached {lens.tolist()}")
    return said


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--batch", type=int, default=4)
    a = ap.parse_args()
    for i, words in enumerate(run(a.steps, a.batch)):
        print(f"request {i}: {len(words)} tokens, the last {words[-8:]}")


if __name__ == "__main__":
    main()
