"""Cases that measure the decode-step operators: attention over a paged cache
for trees of drafted tokens and for selected entries, the accumulated weight
and the eviction it drives, and the verification of drafted tokens.

``run`` computes a case in elementary float32 torch operations, or, with
``own`` set, by the package's public calls.  ``exact`` computes it in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _attn(name, op, **kw):
    c = dict(name=name, op=op, batch=1, next_n=1, tree=False, q_heads=32, kv_heads=8, dim=128,
             len_min=1, len_max=1024, page=64, dtype="bf16", fused_kv=False)
    c.update(kw)
    return c


def listed():
    return [
        # one user, one token, a short chat: latency alone
        _attn("tree_one_token", "tree", len_min=1027, len_max=1027),
        # a serving batch of ragged lengths with three chained drafts each (MTP)
        _attn("tree_mtp_batch", "tree", batch=64, next_n=4, len_min=1, len_max=8192, dtype="f16"),
        # wide trees of drafts: 512 query rows share each cached head
        _attn("tree_wide", "tree", batch=16, next_n=64, tree=True, kv_heads=4, len_min=4000,
              len_max=8192, page=16),
        # two very long contexts, keys and values in one buffer, token-granular pages
        _attn("tree_long", "tree", batch=2, next_n=8, tree=True, dim=64, len_min=163840,
              len_max=163840, page=1, fused_kv=True),
        # the indexer's selection of a decode batch: 2048 entries a row
        dict(name="selected_decode", op="selected", rows=64, top_k=2048, q_heads=32, kv_heads=2,
             dim=128, slots=262144, short=0.1, dtype="bf16"),
        # the selection of an MTP batch over one shared latent-like head
        dict(name="selected_mtp", op="selected", rows=512, top_k=1024, q_heads=16, kv_heads=1,
             dim=128, slots=262144, short=0.25, dtype="f16"),
        # one request's weights after one token
        _attn("weights_one_token", "weights", len_min=2049, len_max=2049, shared=True, accept=False),
        # a batch's weights, each cached head its own, only accepted drafts counted
        _attn("weights_batch", "weights", batch=32, next_n=8, tree=True, len_min=2048, len_max=16384,
              shared=False, accept=True),
        # one request over its budget
        dict(name="evict_one", op="evict", batch=1, next_n=1, accept=False, kv_heads=8, dim=128,
             len_min=5001, len_max=5001, page=64, budget=2048, recent=256, shared=True, dtype="bf16"),
        # a batch evicted head by head after its drafts were verified
        dict(name="evict_batch", op="evict", batch=32, next_n=8, accept=True, kv_heads=8, dim=128,
             len_min=2048, len_max=32768, page=16, budget=4096, recent=512, shared=False, dtype="bf16"),
        # one request's sampled chain against the draft's own probabilities
        dict(name="verify_chain", op="verify", batch=1, next_n=4, tree=False, vocab=32000,
             dtype="f32", draft=True, greedy=0.0),
        # a batch of drafted trees against a large vocabulary, some requests greedy
        dict(name="verify_trees", op="verify", batch=64, next_n=16, tree=True, vocab=131073,
             dtype="bf16", draft=False, greedy=0.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "selected", "weights", "evict", "verify"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("tree", "weights"):
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 6, 8, 16])
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        batch = _log(rng, 1, 64)
        next_n = rng.choice([1, 1, 2, 4, 5, 8, 16, 33, 64])
        most = min(65536, (1 << 28) // (batch * kv * dim), (1 << 34) // (batch * next_n * kv * group * dim))
        hi = max(next_n, _log(rng, 64, max(65, most)))
        c = dict(op=op, batch=batch, next_n=next_n, tree=next_n > 1 and rng.random() < 0.6, q_heads=kv * group,
                 kv_heads=kv, dim=dim, len_min=max(1, hi // rng.choice([1, 2, 16])), len_max=hi,
                 page=rng.choice([1, 7, 16, 32, 64, 100, 128]), dtype=dtype, fused_kv=rng.random() < 0.3)
        if op == "weights":
            c.update(shared=rng.random() < 0.5, accept=rng.random() < 0.5)
        return c
    if op == "selected":
        kv = rng.choice([1, 2, 4])
        dim = rng.choice([64, 96, 128, 256])
        top_k = rng.choice([512, 1024, 2048, _log(rng, 1, 2048)])
        rows = _log(rng, 1, max(2, min(512, (1 << 26) // (top_k * kv * dim))))
        return dict(op=op, rows=rows, top_k=top_k, q_heads=kv * rng.choice([1, 4, 7, 8, 16]), kv_heads=kv,
                    dim=dim, slots=_log(rng, 4096, 131072), short=round(rng.uniform(0, 0.5), 2), dtype=dtype)
    if op == "evict":
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 96, 128, 256])
        batch = _log(rng, 1, 32)
        next_n = rng.choice([1, 4, 8, 16])
        hi = _log(rng, 512, max(513, min(65536, (1 << 27) // (batch * kv * dim))))
        budget = max(16, _log(rng, max(16, hi // 16), hi))
        return dict(op=op, batch=batch, next_n=next_n, accept=rng.random() < 0.6, kv_heads=kv, dim=dim,
                    len_min=max(next_n, hi // 2), len_max=hi, page=rng.choice([1, 7, 16, 64, 100]), budget=budget,
                    recent=rng.choice([0, budget // 8, budget // 2]), shared=rng.random() < 0.5, dtype=dtype)
    next_n = rng.choice([1, 2, 4, 5, 8, 16, 33])
    tree = next_n > 1 and rng.random() < 0.5
    vocab = _log(rng, 1000, 200000)
    batch = _log(rng, 1, max(2, min(128, (1 << 26) // (next_n * vocab))))
    return dict(op=op, batch=batch, next_n=next_n, tree=tree, vocab=vocab, dtype=rng.choice(["bf16", "f16", "f32"]),
                draft=not tree and rng.random() < 0.5, greedy=rng.choice([0.0, 0.3, 1.0]))


# ------------------------------------------------------------------ inputs

def _normal(shape, g, dev, dtype):
    return torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)


def _pages(lens_max, batch, page, g, dev, extra=0):
    """A pool of pages in random order: tables for ``batch`` requests of up
    to ``lens_max`` positions (and one of ``extra`` positions each)."""
    cols, more = -(-lens_max // page), -(-extra // page) if extra else 0
    pages = batch * (cols + more) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = order[:batch * cols].view(batch, cols).contiguous()
    other = order[batch * cols:batch * (cols + more)].view(batch, more).contiguous()
    return pages, table, other


def _lens(case, g, dev):
    lens = torch.randint(case["len_min"], case["len_max"] + 1, (case["batch"],), generator=g, device=dev,
                         dtype=torch.int32)
    lens[0] = case["len_max"]
    if case["batch"] >= 8:
        lens[case["batch"] // 2] = 0    # an idle place of the batch
    return lens


def _caches(slots, case, g, dev):
    dt, h, d = _DT[case["dtype"]], case["kv_heads"], case["dim"]
    if case.get("fused_kv"):
        both = _normal((slots, 2, h, d), g, dev, dt)
        return both[:, 0], both[:, 1]
    return _normal((slots, h, d), g, dev, dt), _normal((slots, h, d), g, dev, dt)


def _accept(batch, n, tree, g, dev):
    """The bits of one accepted path a request: a random node's ancestors."""
    node = torch.randint(0, n, (batch,), generator=g, device=dev)
    return tree.view(batch, n)[torch.arange(batch, device=dev), node].contiguous()


def prepare(case, seed):
    def trees(batch, n, wide, seed):
        """int64 [batch * n]: bit j of row i is set where node j is node i or one
        of its ancestors; the root is node 0, chains without ``wide``."""
        r = np.random.RandomState(seed % (1 << 31))
        rows = np.zeros((batch, n), dtype=np.uint64)
        rows[:, 0] = 1
        at = np.arange(batch)
        for i in range(1, n):
            parent = np.maximum(0, i - 1 - (r.randint(0, 4, batch) if wide else 0)) * np.ones(batch, dtype=np.int64)
            rows[:, i] = rows[at, parent] | (np.uint64(1) << np.uint64(i))
        return torch.from_numpy(rows.reshape(-1).view(np.int64).copy())

    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("tree", "weights"):
        b, n = case["batch"], case["next_n"]
        pages, table, _ = _pages(case["len_max"], b, case["page"], g, dev)
        s["lens"] = _lens(case, g, dev)
        cols = table.shape[1]
        used = (s["lens"].unsqueeze(1) + case["page"] - 1) // case["page"]
        s["table"] = torch.where(torch.arange(cols, device=dev) < used, table, -1)
        s["k"], s["v"] = _caches(pages * case["page"], case, g, dev)
        s["q"] = _normal((b * n, case["q_heads"], case["dim"]), g, dev, _DT[case["dtype"]])
        s["tree"] = trees(b, n, case["tree"], seed).to(dev)
        s["mask"] = s["tree"] if case["tree"] else None
        s["scale"] = case["dim"] ** -0.5
        if op == "weights":
            s["accept"] = _accept(b, n, s["tree"], g, dev) if case["accept"] else None
            s["lse"] = _plain_tree(s)[1]
            s["weights"] = torch.rand((b, 1 if case["shared"] else case["kv_heads"], case["len_max"]), generator=g,
                                      device=dev)
            del s["v"]
    elif op == "selected":
        r, k = case["rows"], case["top_k"]
        s["k"], s["v"] = _caches(case["slots"], case, g, dev)
        s["q"] = _normal((r, case["q_heads"], case["dim"]), g, dev, _DT[case["dtype"]])
        s["idx"] = torch.randint(0, case["slots"], (r, k), generator=g, device=dev, dtype=torch.int32)
        full = torch.rand((r, 1), generator=g, device=dev) >= case["short"]
        count = torch.where(full, k, torch.randint(0, k + 1, (r, 1), generator=g, device=dev))
        s["idx"] = torch.where(torch.arange(k, device=dev) < count, s["idx"], -1)
        s["scale"] = case["dim"] ** -0.5
    elif op == "evict":
        b, n = case["batch"], case["next_n"]
        pages, s["table"], s["new_table"] = _pages(case["len_max"], b, case["page"], g, dev, case["budget"])
        s["lens"] = _lens(case, g, dev)
        s["k"], s["v"] = _caches(pages * case["page"], case, g, dev)
        heads = 1 if case["shared"] else case["kv_heads"]
        s["weights"] = torch.empty((b, heads, case["len_max"]), device=dev).exponential_(generator=g)
        s["accept"] = _accept(b, n, trees(b, n, True, seed).to(dev), g, dev) if case["accept"] else None
    else:
        b, n, vocab = case["batch"], case["next_n"], case["vocab"]
        logits = _normal((b * n, vocab), g, dev, torch.float32).mul_(1.5)
        likely = torch.randint(0, vocab, (b * n, 8), generator=g, device=dev)
        logits.scatter_add_(1, likely, 9 + 2 * torch.randn((b * n, 8), generator=g, device=dev))
        s["logits"] = logits.to(_DT[case["dtype"]])
        s["tree"] = trees(b, n, case["tree"], seed).to(dev)
        s["mask"] = s["tree"] if case["tree"] else None
        s["uniforms"] = torch.rand(b * n, generator=g, device=dev)
        s["noise"] = torch.empty((b, vocab), device=dev).exponential_(generator=g).clamp_(min=1e-20)
        t = 0.6 + 0.6 * torch.rand(b, generator=g, device=dev)
        s["temperature"] = torch.where(torch.rand(b, generator=g, device=dev) < case["greedy"], 0.0, t)
        race = torch.empty((b * n, vocab), device=dev).exponential_(generator=g).log_().neg_()
        if case["draft"]:
            logits += 0.5 * torch.randn(logits.shape, generator=g, device=dev)
            s["draft"] = torch.softmax(logits, 1)
        else:
            s["draft"] = None
        # each draft is a likely token of its parent's row
        proposed = (logits + race).topk(4, 1).indices
        parent = _parents(s["tree"].view(b, n))
        rank = torch.arange(n, device=dev) % (4 if case["tree"] else 1)
        rows = torch.arange(b, device=dev).unsqueeze(1) * n + parent
        s["tokens"] = proposed[rows, rank.expand(b, n)].to(torch.int32).reshape(-1).contiguous()
    return s


# ------------------------------------------------------------- plain forms

def _parents(tree):
    """The highest other bit of each row of [batch, n] trees (0 for the root)."""
    n = tree.shape[1]
    at = torch.arange(n, device=tree.device)
    bits = ((tree.unsqueeze(2) >> at) & 1).bool() & (at < at.unsqueeze(1))
    return torch.where(bits, at, 0).amax(2)


def _visible(s, n):
    """bool [batch, next_n, n]"""
    c, dev = s["case"], s["lens"].device
    at = torch.arange(n, device=dev)
    draft = at - (s["lens"].unsqueeze(1) - c["next_n"])
    bit = (s["tree"].view(c["batch"], c["next_n"], 1) >> draft.clamp(0, 63).unsqueeze(1)) & 1
    draft = draft.unsqueeze(1)
    return (draft < 0) | ((draft < c["next_n"]) & (bit == 1))


def _rows_of(cache, table, page, n):
    at = torch.arange(n, device=table.device)
    slots = table[:, at // page].clamp(min=0).long() * page + at % page
    return cache[slots].float()


def _scores(s):
    c, n = s["case"], s["case"]["len_max"]
    b, h = c["batch"], c["kv_heads"]
    k = _rows_of(s["k"], s["table"], c["page"], n)
    q = s["q"].float().view(b, c["next_n"], h, -1, c["dim"])
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(b, h, -1, c["dim"]), k.permute(0, 2, 3, 1))
    x = (x * s["scale"]).view(b, h, c["next_n"], -1, n)
    return x.masked_fill_(~_visible(s, n).view(b, 1, c["next_n"], 1, n), -math.inf)


def _softmax(x):
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (x - top).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(torch.where(total == 0, 1.0, total)), (top + total.log()).squeeze(-1)


def _plain_tree(s):
    c = s["case"]
    b, h, n = c["batch"], c["kv_heads"], c["len_max"]
    p, lse = _softmax(_scores(s))
    lse = lse.permute(0, 2, 1, 3).reshape(b * c["next_n"], -1)
    v = _rows_of(s["v"], s["table"], c["page"], n).permute(0, 2, 1, 3)
    out = torch.matmul(p.view(b, h, -1, n), v).view(b, h, c["next_n"], -1, c["dim"])
    return out.permute(0, 2, 1, 3, 4).reshape(s["q"].shape).to(s["q"].dtype), lse.contiguous()


def _plain_selected(s):
    c, idx = s["case"], s["idx"]
    r, h = c["rows"], c["kv_heads"]
    at = idx.clamp(min=0).long()
    q = s["q"].float().view(r, h, -1, c["dim"])
    x = torch.matmul(q, s["k"][at].float().permute(0, 2, 3, 1)) * s["scale"]
    p, lse = _softmax(x.masked_fill_((idx < 0).view(r, 1, 1, -1), -math.inf))
    out = torch.matmul(p, s["v"][at].float().permute(0, 2, 1, 3))
    return out.reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(r, -1)


def _plain_weights(s):
    c, n = s["case"], s["case"]["len_max"]
    b, h, t = c["batch"], c["kv_heads"], c["next_n"]
    lse = s["lse"].view(b, t, h, -1).permute(0, 2, 1, 3).unsqueeze(-1)
    p = torch.where(lse == -math.inf, 0.0, (_scores(s) - lse).exp_())
    if s["accept"] is not None:
        took = (s["accept"].unsqueeze(1) >> torch.arange(t, device=p.device)) & 1
        p = p * took.view(b, 1, t, 1, 1)
    s["weights"] += p.sum((1, 2, 3)).unsqueeze(1) if c["shared"] else p.sum((2, 3))
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    b, n, h, m = c["batch"], c["len_max"], c["kv_heads"], c["budget"]
    dev = s["lens"].device
    at = torch.arange(n, device=dev)
    alive = at < s["lens"].unsqueeze(1)
    if s["accept"] is not None:
        draft = at - (s["lens"].unsqueeze(1) - c["next_n"])
        alive &= (draft < 0) | (((s["accept"].unsqueeze(1) >> draft.clamp(0, 63)) & 1) == 1)
    count = alive.sum(1, keepdim=True)
    late = alive.sum(1, keepdim=True) - alive.cumsum(1) < c["recent"]     # the last survivors
    w = s["weights"]
    rank = torch.where(late.unsqueeze(1), math.inf, w).masked_fill(~alive.unsqueeze(1), -math.inf)
    best = rank.sort(dim=2, descending=True, stable=True).indices[:, :, :m]
    m_row = count.clamp(max=m).unsqueeze(2)
    there = torch.arange(best.shape[2], device=dev) < m_row
    kept = torch.where(there, best, n).sort(dim=2).values
    there = kept < n
    new = torch.full((b, w.shape[1], m), -1, dtype=torch.int32, device=dev)
    new[:, :, :kept.shape[2]] = torch.where(there, kept, -1).to(torch.int32)
    out_w = torch.zeros_like(w)
    out_w[:, :, :kept.shape[2]] = torch.where(there, w.gather(2, kept.clamp(max=n - 1)), 0.0)
    # rows to their new pages
    bi, hi, ji = there.expand(b, w.shape[1], -1).nonzero(as_tuple=True)
    p = kept[bi, hi, ji]
    src = s["table"][bi, p // c["page"]].long() * c["page"] + p % c["page"]
    dst = s["new_table"][bi, ji // c["page"]].long() * c["page"] + ji % c["page"]
    if c["shared"]:
        s["k"][dst], s["v"][dst] = s["k"][src], s["v"][src]
    else:
        s["k"][dst, hi], s["v"][dst, hi] = s["k"][src, hi], s["v"][src, hi]
    return new, count.squeeze(1).clamp(max=m).to(torch.int32), out_w, s["k"], s["v"]


def _plain_verify(s):
    c = s["case"]
    b, n, vocab = c["batch"], c["next_n"], c["vocab"]
    dev = s["logits"].device
    x = s["logits"].float().view(b, n, vocab)
    t = s["temperature"].view(b, 1, 1)
    top = x.amax(2, keepdim=True)
    at = torch.arange(vocab, device=dev)
    first = torch.where(x == top, at, vocab).amin(2, keepdim=True)
    p = ((x - top) / torch.where(t > 0, t, 1.0)).exp_()
    p = p / p.sum(2, keepdim=True)
    p = torch.where(t > 0, p, (at == first).float())
    tree, token = s["tree"].view(b, n), s["tokens"].view(b, n).long()
    node = torch.arange(n, device=dev)
    parent = _parents(tree)
    bi = torch.arange(b, device=dev)
    older = (parent.unsqueeze(2) == parent.unsqueeze(1)) & (node < node.unsqueeze(1)) & (node > 0)
    again = (older & (token.unsqueeze(2) == token.unsqueeze(1))).any(2)
    mine = torch.where(again, 0.0, p[bi.unsqueeze(1), parent, token])
    u = s["uniforms"].view(b, n)
    if s["draft"] is not None:
        q = s["draft"].view(b, n, vocab)
        passed = u * q[bi.unsqueeze(1), parent, token] < mine
    else:
        passed = u * (1 - (older * mine.unsqueeze(1)).sum(2)) < mine
    chosen = passed & ~(older & passed.unsqueeze(1)).any(2)
    chosen[:, 0] = True
    above = ((tree.unsqueeze(2) >> node) & 1).bool()
    took = (chosen.unsqueeze(1) | ~above).all(2)
    last = torch.where(took, node, 0).amax(1)
    rest = p[bi, last].clone()
    below = (parent == last.unsqueeze(1)) & (node > 0)
    if s["draft"] is not None:
        rest = torch.where(below.any(1, keepdim=True), (rest - q[bi, last]).clamp(min=0), rest)
    else:
        gone = torch.zeros((b, vocab + 1), dtype=torch.bool, device=dev)
        gone.scatter_(1, torch.where(below, token, vocab), True)
        rest = rest.masked_fill(gone[:, :vocab], 0.0)
    race = rest / s["noise"]
    best = race.amax(1, keepdim=True)
    next_token = torch.where((race == best) & (best > 0), at, vocab).amin(1)
    next_token = torch.where(next_token == vocab, -1, next_token)
    path = torch.where(took, node, n).sort(1).values
    mask = (took.long() << node).sum(1)
    return (took.sum(1).to(torch.int32) - 1, torch.where(path == n, -1, path).to(torch.int32),
            next_token.to(torch.int32), mask)


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"tree": _plain_tree, "selected": _plain_selected, "weights": _plain_weights,
                "evict": _plain_evict, "verify": _plain_verify}[op](s)
    import sparse_attention_top_gb300 as gb
    if op == "tree":
        return gb.tree_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], page_size=c["page"],
                                 next_n=c["next_n"], tree_mask=s["mask"], return_lse=True)
    if op == "selected":
        return gb.selected_attention(s["q"], s["k"], s["v"], s["idx"], return_lse=True)
    if op == "weights":
        return gb.accumulate_cache_weights(s["q"], s["k"], s["lse"], s["table"], s["lens"], s["weights"],
                                           page_size=c["page"], next_n=c["next_n"], tree_mask=s["mask"],
                                           accept_mask=s["accept"])
    if op == "evict":
        return gb.evict_cache(s["weights"], s["k"], s["v"], s["table"], s["lens"], s["new_table"], c["budget"],
                              recent=c["recent"], page_size=c["page"], next_n=c["next_n"],
                              accept_mask=s["accept"]) + (s["k"], s["v"])
    return gb.verify_drafts(s["logits"], s["tokens"], s["uniforms"], s["noise"], next_n=c["next_n"],
                            tree_mask=s["mask"], temperature=s["temperature"], draft_probs=s["draft"])


# --------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    es = 4 if case["dtype"] == "f32" else 2
    if op == "verify":
        b, n, v = case["batch"], case["next_n"], case["vocab"]
        return {"bytes": b * n * v * es + b * v * 4 * (2 if case["draft"] else 1) + b * n * 24, "flops": 4 * b * n * v}
    if op == "selected":
        pairs = case["rows"] * case["top_k"] * (1 - case["short"] / 2)
        row = case["rows"] * case["q_heads"] * case["dim"]
        return {"bytes": pairs * (2 * case["kv_heads"] * case["dim"] * es + 4) + 2 * row * es,
                "flops": 4 * pairs * case["q_heads"] * case["dim"]}
    mean = case["len_max"] if case["batch"] == 1 else (case["len_min"] + case["len_max"]) / 2
    tokens = mean * case["batch"]
    wide = case["kv_heads"] * case["dim"] * es
    if op == "evict":
        heads = 1 if case["shared"] else case["kv_heads"]
        kept = min(mean, case["budget"]) * case["batch"]
        return {"bytes": tokens * heads * 4 + kept * (4 * wide + 8 * heads), "flops": tokens * heads}
    rows = case["batch"] * case["next_n"] * case["q_heads"]
    pairs = rows * mean
    if op == "weights":
        heads = 1 if case["shared"] else case["kv_heads"]
        return {"bytes": tokens * (wide + 8 * heads) + rows * (case["dim"] * es + 4), "flops": 2 * pairs * case["dim"]}
    return {"bytes": tokens * 2 * wide + rows * (2 * case["dim"] * es + 4), "flops": 4 * pairs * case["dim"]}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions, request by request, in 64 bits."""
    def seen(s, i):
        """Request i's slots in order, and which of them its rows see."""
        c = s["case"]
        length, n = int(s["lens"][i]), c["next_n"]
        slots = [int(p) * c["page"] + o for p in s["table"][i].tolist() for o in range(c["page"])][:length]
        ctx = length - n
        see = torch.ones((n, len(slots)), dtype=torch.bool)
        for t in range(n):
            bits = int(s["tree"][i * n + t]) & ((1 << 64) - 1)
            for j in range(n):
                if 0 <= ctx + j < len(slots):
                    see[t, ctx + j] = bool(bits >> j & 1)
        return torch.tensor(slots, dtype=torch.long, device=s["lens"].device), see.to(s["lens"].device)

    def group64(q, k, see, scale):
        """Scaled products of [rows, group, dim] queries with [n, dim] keys."""
        x = torch.einsum("tgd,nd->tgn", q.double(), k.double()) * scale
        return x.masked_fill(~see.unsqueeze(1), -math.inf)

    def attend64(q, k, v, see, scale):
        if k.shape[0] == 0:
            return torch.zeros(q.shape, dtype=torch.float64, device=q.device), \
                torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
        x = group64(q, k, see, scale)
        lse = torch.logsumexp(x, 2)
        p = torch.where(lse.unsqueeze(2) == -math.inf, 0.0, (x - lse.unsqueeze(2)).exp())
        return torch.einsum("tgn,nd->tgd", p, v.double()), lse

    def attention(s):
        c = s["case"]
        n, g = c["next_n"], c["q_heads"] // c["kv_heads"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
        for i in range(c["batch"]):
            slots, see = seen(s, i)
            rows = slice(i * n, i * n + n)
            for h in range(c["kv_heads"]):
                heads = slice(h * g, h * g + g)
                out[rows, heads], lse[rows, heads] = attend64(s["q"][rows, heads], s["k"][slots, h], s["v"][slots, h],
                                                               see, c["dim"] ** -0.5)
        return out, lse

    def selected(s):
        c = s["case"]
        g = c["q_heads"] // c["kv_heads"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
        for r in range(c["rows"]):
            slots = s["idx"][r][s["idx"][r] >= 0].long()
            see = torch.ones((1, slots.numel()), dtype=torch.bool, device=slots.device)
            for h in range(c["kv_heads"]):
                heads = slice(h * g, h * g + g)
                out[r:r + 1, heads], lse[r:r + 1, heads] = attend64(s["q"][r:r + 1, heads], s["k"][slots, h],
                                                                     s["v"][slots, h], see, c["dim"] ** -0.5)
        return out, lse

    def weights(s):
        c = s["case"]
        n, g = c["next_n"], c["q_heads"] // c["kv_heads"]
        w = s["weights"].double()
        for i in range(c["batch"]):
            slots, see = seen(s, i)
            if not slots.numel():
                continue
            bits = int(s["accept"][i]) & ((1 << 64) - 1) if s["accept"] is not None else (1 << 64) - 1
            for h in range(c["kv_heads"]):
                x = group64(s["q"][i * n:i * n + n, h * g:h * g + g], s["k"][slots, h], see, c["dim"] ** -0.5)
                lse = s["lse"][i * n:i * n + n, h * g:h * g + g].double().unsqueeze(2)
                p = torch.where(lse == -math.inf, 0.0, (x - lse).exp()).sum(1)
                for t in range(n):
                    if bits >> t & 1:
                        w[i, 0 if c["shared"] else h, :slots.numel()] += p[t]
        return w

    def evict(s):
        c = s["case"]
        m, n = c["budget"], c["next_n"]
        kept = torch.full((c["batch"], s["weights"].shape[1], m), -1, dtype=torch.int32)
        lens = torch.zeros(c["batch"], dtype=torch.int32)
        out_w = torch.zeros_like(s["weights"], dtype=torch.float64)
        k, v = s["k"].clone(), s["v"].clone()
        for i in range(c["batch"]):
            length = int(s["lens"][i])
            alive = list(range(length))
            if s["accept"] is not None:
                bits = int(s["accept"][i]) & ((1 << 64) - 1)
                alive = [p for p in alive if p < length - n or bits >> (p - length + n) & 1]
            lens[i] = min(m, len(alive))
            old, new = s["table"][i].tolist(), s["new_table"][i].tolist()
            for h in range(s["weights"].shape[1]):
                keep = alive
                if len(alive) > m:
                    cut = len(alive) - c["recent"]
                    w = s["weights"][i, h].cpu().numpy()
                    others = np.array(alive[:cut])
                    best = others[np.argsort(-w[others].astype(np.float64), kind="stable")[:m - c["recent"]]]
                    keep = sorted(best.tolist()) + alive[cut:]
                if not keep:
                    continue
                at = torch.tensor(keep)
                kept[i, h, :len(keep)] = at.to(torch.int32)
                out_w[i, h, :len(keep)] = s["weights"][i, h][at.to(k.device)].double()
                src = torch.tensor([old[p // c["page"]] * c["page"] + p % c["page"] for p in keep], device=k.device)
                dst = torch.tensor([new[j // c["page"]] * c["page"] + j % c["page"] for j in range(len(keep))],
                                   device=k.device)
                for x, y in ((k, s["k"]), (v, s["v"])):
                    if c["shared"]:
                        x[dst] = y[src]
                    else:
                        x[dst, h] = y[src, h]
        return kept, lens, out_w, k, v

    def verify(s):
        c = s["case"]
        b, n, vocab = c["batch"], c["next_n"], c["vocab"]
        accepted, follow, masks = [], [], []
        paths = torch.full((b, n), -1, dtype=torch.int32)
        token, u = s["tokens"].tolist(), s["uniforms"].tolist()
        for i in range(b):
            t = float(s["temperature"][i])
            parent = [0] * n
            for j in range(1, n):
                parent[j] = max(a for a in range(j) if (int(s["tree"][i * n + j]) & ((1 << 64) - 1)) >> a & 1)
            cur, path = 0, [0]
            while True:
                x = s["logits"][i * n + cur].double()
                if t > 0:
                    rest = torch.softmax(x / t, 0)
                else:
                    rest = torch.zeros_like(x)
                    rest[int((x == x.max()).nonzero()[0])] = 1
                q = s["draft"][i * n + cur].double() if s["draft"] is not None else None
                mass, found = 1.0, None
                for j in range(cur + 1, n):
                    if parent[j] != cur:
                        continue
                    at = token[i * n + j]
                    have = float(rest[at])
                    if u[i * n + j] * (float(q[at]) if q is not None else mass) < have:
                        found = j
                        break
                    if q is not None:
                        rest = (rest - q).clamp(min=0)
                    else:
                        mass -= have
                        rest[at] = 0
                if found is None:
                    break
                cur = found
                path.append(cur)
            race = rest / s["noise"][i].double()
            follow.append(int((race == race.max()).nonzero()[0]) if float(race.max()) > 0 else -1)
            accepted.append(len(path) - 1)
            paths[i, :len(path)] = torch.tensor(path, dtype=torch.int32)
            bits = sum(1 << j for j in path)
            masks.append(bits - (1 << 64) if bits >> 63 else bits)
        return (torch.tensor(accepted, dtype=torch.int32), paths, torch.tensor(follow, dtype=torch.int32),
                torch.tensor(masks, dtype=torch.int64))

    return {"tree": attention, "selected": selected, "weights": weights, "evict": evict,
            "verify": verify}[case["op"]](prepare(case, seed))
