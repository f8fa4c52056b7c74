"""Cases that measure the operators from the prompt to a 4-bit cache: norms and
rotation of queries and keys with the cache write in the same pass (16-bit and
4-bit), reading a 4-bit cache back, attention over it, and attention over
packed prompts.

``run`` computes a case in elementary float32 torch operations (64 bits for
angles and for what is next to a rounding border), or, with ``own`` set, by the
package's public calls.  ``exact`` computes it in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _rotate(name, op, **kw):
    c = dict(name=name, op=op, tokens=1, context=0, q_heads=32, kv_heads=8, dim=128, rotary=128, interleaved=False,
             norm=True, far=131072, pad=0, dtype="bf16")
    c.update(kw)
    return c


def _attn(name, **kw):
    c = dict(name=name, op="tree4", batch=1, next_n=1, tree=False, q_heads=32, kv_heads=8, dim=128, len_min=1,
             len_max=1024, page=64, dtype="bf16")
    c.update(kw)
    return c


def _prompt(name, **kw):
    c = dict(name=name, op="prompt", batch=1, q_heads=32, kv_heads=8, dim=128, len_min=1, len_max=1024, context=0,
             tail=0, dtype="bf16")
    c.update(kw)
    return c


def listed():
    return [
        # a speculative decode batch: 64 requests x 4 tokens into a 16-bit cache, some places of the batch idle
        _rotate("rotate_decode", "rotate", tokens=256, pad=8),
        # a long prompt into a 16-bit cache, rotation of neighbouring pairs over half of each head
        _rotate("rotate_prompt", "rotate", tokens=16001, rotary=64, interleaved=True, dtype="f16"),
        # one user, one token into a 4-bit cache, and the last window of it read back
        _rotate("quantise_one", "quantise", tokens=1, context=127),
        # a chunk of a prompt into a 4-bit cache, and the whole context so far read back for the chunk's attention
        _rotate("quantise_prompt", "quantise", tokens=8192, context=24577),
        # one user, one token, a short chat over a 4-bit cache: latency alone
        _attn("tree4_one", len_min=1027, len_max=1027),
        # a serving batch of ragged lengths with three chained drafts each
        _attn("tree4_batch", batch=64, next_n=4, len_min=1, len_max=8192, dtype="f16"),
        # few very long contexts with trees of drafts, small pages
        _attn("tree4_long", batch=4, next_n=8, tree=True, kv_heads=4, len_min=131000, len_max=131072, page=16),
        # the indexer's selection for one token
        dict(name="selected4_one", op="selected4", rows=1, top_k=2048, q_heads=32, kv_heads=8, dim=128, slots=65536,
             short=0.0, dtype="bf16"),
        # the indexer's selection of a decode batch
        dict(name="selected4_decode", op="selected4", rows=64, top_k=2048, q_heads=32, kv_heads=2, dim=128,
             slots=262144, short=0.1, dtype="f16"),
        # a batch of short chats packed into one call, some rows of the buffer behind the last
        _prompt("prompt_batch", batch=16, len_min=1, len_max=2048, tail=37, dtype="f16"),
        # one long document
        _prompt("prompt_long", len_min=10007, len_max=10007),
        # a chunk of a long prompt over the context before it, narrow heads
        _prompt("prompt_chunk", batch=2, kv_heads=4, dim=64, len_min=1500, len_max=2048, context=16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "quantise", "tree4", "tree4", "selected4", "prompt", "prompt"])
    dtype = rng.choice(["bf16", "f16"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16])
    if op in ("rotate", "quantise"):
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        tokens = _log(rng, 1, min(16384, (1 << 26) // ((group + 2) * kv * dim)))
        context = _log(rng, 1, min(32768, (1 << 25) // (kv * dim)))
        return dict(op=op, tokens=tokens, context=context if op == "quantise" else 0, q_heads=kv * group,
                    kv_heads=kv, dim=dim, rotary=rng.choice([dim, dim, dim // 32 * 16]), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.7, far=rng.choice([4096, 131072, 1 << 20]), pad=rng.choice([0, 0, 1, tokens // 9]),
                    dtype=dtype)
    if op == "tree4":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        batch = _log(rng, 1, 64)
        next_n = rng.choice([1, 1, 2, 4, 5, 8, 16, 33])
        most = min(131072, (1 << 28) // (batch * kv * dim), (1 << 34) // (batch * next_n * kv * group * dim))
        hi = max(next_n, _log(rng, 64, max(65, most)))
        return dict(op=op, batch=batch, next_n=next_n, tree=next_n > 1 and rng.random() < 0.6, q_heads=kv * group,
                    kv_heads=kv, dim=dim, len_min=max(1, hi // rng.choice([1, 2, 16])), len_max=hi,
                    page=rng.choice([1, 7, 16, 32, 64, 100, 128]), dtype=dtype)
    if op == "selected4":
        dim = rng.choice([64, 96, 128, 256])
        top_k = rng.choice([512, 1024, 2048, _log(rng, 1, 2048)])
        rows = _log(rng, 1, max(2, min(512, (1 << 26) // (top_k * kv * dim))))
        return dict(op=op, rows=rows, top_k=top_k, q_heads=kv * rng.choice([1, 4, 7, 8, 16]), kv_heads=kv, dim=dim,
                    slots=_log(rng, 4096, 131072), short=round(rng.uniform(0, 0.5), 2), dtype=dtype)
    dim = rng.choice([64, 80, 96, 128, 128, 256])
    batch = _log(rng, 1, 32)
    hi = _log(rng, 1, max(2, int(((1 << 36) / (batch * kv * group * dim)) ** 0.5)))
    context = rng.choice([0, 0, _log(rng, 1, max(2, min(16384, (1 << 36) // (batch * kv * group * dim * hi))))])
    return dict(op="prompt", batch=batch, q_heads=kv * group, kv_heads=kv, dim=dim, len_min=max(1, hi // rng.choice([1, 2, 16])),
                len_max=hi, context=context, tail=rng.choice([0, 0, 5]), dtype=dtype)


# ------------------------------------------------------- rows of a 4-bit cache

def _areas(dim):
    """Bytes of a row's codes (of keys, and as many of values) and scales."""
    return -(-dim // 32) * 16, 8 if dim <= 128 else 16


def _pack(k, v):
    """[..., dim] keys and values as rows of a 4-bit cache (uint8)."""
    dim = k.shape[-1]
    c, s = _areas(dim)
    row = torch.zeros(k.shape[:-1] + (2 * c + 2 * s,), dtype=torch.uint8, device=k.device)
    for i, x in enumerate((k, v)):
        scale, code = _quantise(x, 1.0)
        bits = _e4m3_bits(scale)
        code = code.to(torch.int64).view(code.shape[:-2] + (-1, 4, 2))
        mag, sign = code.abs(), (code < 0).long()
        at = torch.arange(4, device=k.device)
        word = (mag[..., 0] << (4 * at)) | (mag[..., 1] << (4 * at + 16))
        word |= (sign[..., 0] << ((4 * at + 15) % 32)) | (sign[..., 1] << ((4 * at + 31) % 32))
        word = word.sum(-1)
        codes = (word.unsqueeze(-1) >> (8 * at)).bitwise_and(255).to(torch.uint8).flatten(-2)
        row[..., i * c:i * c + dim // 2] = codes
        row[..., 2 * c + i * s:2 * c + i * s + dim // 16] = bits
    return row


def _quantise(x, unit):
    """Scales [..., dim // 16] in units of `unit` and codes [..., dim // 16, 16], in 64 bits."""
    x = x.double().unflatten(-1, (-1, 16)) / unit
    top = torch.where(x.isnan(), 0.0, x.abs()).amax(-1)
    scale = _e4m3((top / top.new_full((1,), 7.0)).clamp(max=448.0))     # (a scalar would be multiplied by 1/7)
    code = torch.where(scale.unsqueeze(-1) > 0, x / torch.where(scale > 0, scale, 1.0).unsqueeze(-1), 0.0)
    return scale, code.round().clamp(-7, 7)


def _exponent(x):
    """floor(log2 x) of normal 64-bit numbers, at least -6."""
    return ((x.view(torch.int64) >> 52) - 1023).clamp(min=-6)


def _e4m3(x):
    """x >= 0 rounded to the nearest 8-bit number of 4 exponent and 3 mantissa bits (ties to even)."""
    step = (_exponent(x) - 3 + 1023 << 52).view(torch.float64)
    return ((x / step).round() * step).clamp(max=448.0)


def _e4m3_bits(x):
    e = _exponent(x)
    m = x / (e - 3 + 1023 << 52).view(torch.float64)       # 8..15, or below 8 in the lowest binade
    return (e + 6) * 8 + m.long()


def _unpack(row, dim):
    """Keys and values [..., dim] (float32) of the rows of a 4-bit cache."""
    c, s = _areas(dim)
    got = []
    for i in range(2):
        word = row[..., i * c:i * c + dim // 2].contiguous().view(torch.int32)
        at = torch.arange(4, device=row.device, dtype=torch.int32)
        w = word.unsqueeze(-1)
        code = torch.stack([(w >> (4 * at)) & 7, (w >> (4 * at + 16)) & 7], -1)
        sign = torch.stack([(w >> ((4 * at + 15) % 32)) & 1, (w >> ((4 * at + 31) % 32)) & 1], -1)
        code = torch.where(sign == 1, -code, code).flatten(-3)
        bits = row[..., 2 * c + i * s:2 * c + i * s + dim // 16].int() & 127
        e, m = bits >> 3, (bits & 7).float()
        scale = torch.where(e > 0, (1 + m / 8) * ((e + 120) << 23).view(torch.float32), m / 512)
        got.append((code.unflatten(-1, (-1, 16)).float() * scale.unsqueeze(-1)).flatten(-2))
    return got


# ------------------------------------------------------------------ inputs

def _normal(shape, g, dev, dtype):
    return torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)


def _lens(case, g, dev):
    """Lengths spread evenly over their range, in random order."""
    b = case["batch"]
    lens = torch.linspace(case["len_max"], case["len_min"], b, dtype=torch.float64).int().to(dev)
    if b >= 8:
        lens[b // 2] = 0    # an idle place of the batch
    return lens[torch.randperm(b, generator=g, device=dev)].contiguous()


def _rows(slots, case, g, dev):
    """A 4-bit cache: keys with channels of their own sizes, values around one."""
    shape = (slots, case["kv_heads"], case["dim"])
    size = torch.exp(0.5 * _normal(shape[1:], g, dev, torch.float32))
    return _pack(_normal(shape, g, dev, torch.float32) * size, _normal(shape, g, dev, torch.float32))


def prepare(case, seed):
    def trees(batch, n, wide):
        """int64 [batch * n]: bit j of row i is set where node j is node i or one
        of its ancestors; the root is node 0, chains without ``wide``."""
        back = torch.randint(0, 4, (n, batch), generator=g, device=dev).cpu()
        rows = torch.zeros((batch, n), dtype=torch.int64)
        rows[:, 0] = 1
        for i in range(1, n):
            parent = (i - 1 - (back[i] if wide else 0 * back[i])).clamp(min=0)
            rows[:, i] = rows.gather(1, parent.unsqueeze(1)).squeeze(1) | (1 << i)
        return rows.view(-1)

    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, s, dt = case["op"], {"case": case}, _DT[case["dtype"]]
    dim, kv, qh = case["dim"], case["kv_heads"], case["q_heads"]
    if op in ("rotate", "quantise"):
        # queries, keys and values as one projection leaves them
        n, width = case["tokens"], qh + 2 * kv
        both = _normal((n, width, dim), g, dev, dt)
        s["q"], s["k"], s["v"] = both[:, :qh], both[:, qh:qh + kv], both[:, qh + kv:]
        first = case["far"] - n - 1
        s["positions"] = torch.arange(n, device=dev, dtype=torch.int32) + max(0, first)
        pool = n + case["context"] + 17
        order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        s["slots"] = order[:n].clone()
        if case["pad"]:
            s["slots"][n - min(n, case["pad"]):] = -1
        half = case["rotary"] // 2
        s["freq"] = (1e4 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)).float()
        s["wq"] = s["wk"] = None
        if case["norm"]:
            s["wq"], s["wk"] = (1 + 0.1 * _normal((2, dim), g, dev, torch.float32)).to(dt)
        if op == "rotate":
            s["k_cache"], s["v_cache"] = torch.zeros((2, pool, kv, dim), dtype=dt, device=dev)
        else:
            s["cache"] = _rows(pool, case, g, dev)
            s["read"] = order[:n + case["context"]].clone()     # the earlier context's slots after the new ones
    elif op == "tree4":
        b, n, page = case["batch"], case["next_n"], case["page"]
        s["lens"] = _lens(case, g, dev)
        cols = -(-case["len_max"] // page)
        pages = b * cols + 3
        table = torch.randperm(pages, generator=g, device=dev)[:b * cols].to(torch.int32).view(b, cols)
        used = (s["lens"].unsqueeze(1) + page - 1) // page
        s["table"] = torch.where(torch.arange(cols, device=dev) < used, table, -1)
        s["cache"] = _rows(pages * page, case, g, dev)
        s["q"] = _normal((b * n, qh, dim), g, dev, dt)
        s["tree"] = trees(b, n, case["tree"]).to(dev)
        s["mask"] = s["tree"] if case["tree"] else None
    elif op == "selected4":
        r, k = case["rows"], case["top_k"]
        s["cache"] = _rows(case["slots"], case, g, dev)
        s["q"] = _normal((r, qh, dim), g, dev, dt)
        idx = torch.randint(0, case["slots"], (r, k), generator=g, device=dev, dtype=torch.int32)
        full = torch.rand((r, 1), generator=g, device=dev) >= case["short"]
        count = torch.where(full, k, torch.randint(0, k + 1, (r, 1), generator=g, device=dev))
        s["idx"] = torch.where(torch.arange(k, device=dev) < count, idx, -1)
    else:
        lens = _lens(case, g, dev)
        longer = torch.linspace(case["context"] // 2, case["context"], case["batch"], dtype=torch.float64).int().to(dev)
        klens = lens + longer
        s["cu"] = torch.nn.functional.pad(lens.cumsum(0, dtype=torch.int32), (1, 0))
        s["cu_k"] = torch.nn.functional.pad(klens.cumsum(0, dtype=torch.int32), (1, 0))
        rows, keys = int(s["cu"][-1]) + case["tail"], int(s["cu_k"][-1]) + case["tail"]
        s["q"] = _normal((rows, qh, dim), g, dev, dt)
        s["k"], s["v"] = _normal((keys, kv, dim), g, dev, dt), _normal((keys, kv, dim), g, dev, dt)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(s["q"].shape[:2], device=dev)
    return s


# ------------------------------------------------------------- plain forms

def _turned(x, w, s, wide):
    """Norm and rotation of [tokens, heads, dim]; `wide`: in 64 bits."""
    c = s["case"]
    x = x.double() if wide else x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.to(x.dtype)
    if not c["rotary"]:
        return x
    angle = s["positions"].double().unsqueeze(1) * s["freq"].double()
    cos, sin = (f(angle).to(x.dtype).unsqueeze(1) for f in (torch.cos, torch.sin))
    head, rest = x[..., :c["rotary"]], x[..., c["rotary"]:]
    if c["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head.chunk(2, -1)
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, rest], -1)


def _plain_rotate(s):
    dt = s["q"].dtype
    at = s["slots"] >= 0
    where = s["slots"][at].long()
    s["k_cache"][where] = _turned(s["k"], s["wk"], s, False).to(dt)[at]
    s["v_cache"][where] = s["v"][at]
    return _turned(s["q"], s["wq"], s, False).to(dt), s["k_cache"], s["v_cache"]


def _plain_quantise(s):
    dt = s["q"].dtype
    at = s["slots"] >= 0
    s["cache"][s["slots"][at].long()] = _pack(_turned(s["k"], s["wk"], s, True), s["v"])[at]
    q = _turned(s["q"], s["wq"], s, False).to(dt)
    k, v = _unpack(s["cache"][s["read"].clamp(min=0).long()], s["case"]["dim"])
    none = (s["read"] < 0).view(-1, 1, 1)
    return q, k.masked_fill(none, 0.0).to(dt), v.masked_fill(none, 0.0).to(dt)


def _softmax(x):
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(torch.where(total == 0, 1.0, total)), (top + total.log()).squeeze(-1)


def _plain_tree(s):
    c = s["case"]
    b, h, n, t, page = c["batch"], c["kv_heads"], c["len_max"], c["next_n"], c["page"]
    at = torch.arange(n, device=s["q"].device)
    slots = s["table"][:, at // page].clamp(min=0).long() * page + at % page
    k, v = _unpack(s["cache"][slots], c["dim"])
    q = s["q"].float().view(b, t, h, -1, c["dim"]).permute(0, 2, 1, 3, 4).reshape(b, h, -1, c["dim"])
    x = (torch.matmul(q, k.permute(0, 2, 3, 1)) * c["dim"] ** -0.5).view(b, h, t, -1, n)
    draft = at - (s["lens"].unsqueeze(1) - t)
    bit = (s["tree"].view(b, t, 1) >> draft.clamp(0, 63).unsqueeze(1)) & 1
    draft = draft.unsqueeze(1)
    sees = (draft < 0) | ((draft < t) & (bit == 1))
    p, lse = _softmax(x.masked_fill_(~sees.view(b, 1, t, 1, n), -math.inf))
    out = torch.matmul(p.view(b, h, -1, n), v.permute(0, 2, 1, 3)).view(b, h, t, -1, c["dim"])
    return (out.permute(0, 2, 1, 3, 4).reshape(s["q"].shape).to(s["q"].dtype),
            lse.permute(0, 2, 1, 3).reshape(b * t, -1).contiguous())


def _plain_selected(s):
    c, idx = s["case"], s["idx"]
    r, h = c["rows"], c["kv_heads"]
    k, v = _unpack(s["cache"][idx.clamp(min=0).long()], c["dim"])
    q = s["q"].float().view(r, h, -1, c["dim"])
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * c["dim"] ** -0.5
    p, lse = _softmax(x.masked_fill_((idx < 0).view(r, 1, 1, -1), -math.inf))
    out = torch.matmul(p, v.permute(0, 2, 1, 3))
    return out.reshape(s["q"].shape).to(s["q"].dtype), lse.reshape(r, -1)


def _plain_prompt(s):
    """Sequences padded to the longest."""
    c, dev = s["case"], s["q"].device
    b, h, d = c["batch"], c["kv_heads"], c["dim"]
    n, m = c["len_max"], c["len_max"] + c["context"]
    lens, klens = s["cu"].diff(), s["cu_k"].diff()
    t, j = torch.arange(n, device=dev), torch.arange(m, device=dev)
    rows = (s["cu"][:-1].unsqueeze(1) + t).clamp(max=s["q"].shape[0] - 1).long()
    keys = (s["cu_k"][:-1].unsqueeze(1) + j).clamp(max=s["k"].shape[0] - 1).long()
    q = s["q"][rows].float().view(b, n, h, -1, d).permute(0, 2, 3, 1, 4)
    k, v = (s[x][keys].float().permute(0, 2, 1, 3).unsqueeze(2) for x in "kv")
    x = torch.matmul(q, k.transpose(3, 4)).mul_(d ** -0.5)
    last = t + (klens - lens).unsqueeze(1)
    sees = (j <= last.unsqueeze(2)) & (j < klens.view(b, 1, 1))
    p, lse = _softmax(x.masked_fill_(~sees.view(b, 1, 1, n, m), -math.inf))
    out = torch.matmul(p, v).permute(0, 3, 1, 2, 4).reshape(b, n, -1, d)
    there = t < lens.unsqueeze(1)
    s["out"][rows[there]] = out[there].to(s["q"].dtype)
    s["lse"][rows[there]] = lse.permute(0, 3, 1, 2).reshape(b, n, -1)[there]
    return s["out"], s["lse"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"rotate": _plain_rotate, "quantise": _plain_quantise, "tree4": _plain_tree,
                "selected4": _plain_selected, "prompt": _plain_prompt}[op](s)
    import sparse_attention_top_gb300 as gb
    if op == "rotate":
        q = gb.rotate_and_cache(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freq"], s["k_cache"],
                                s["v_cache"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6,
                                interleaved=c["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    if op == "quantise":
        q = gb.rotate_and_cache_int4(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freq"], s["cache"],
                                     q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, interleaved=c["interleaved"])
        return (q,) + tuple(gb.read_cache_int4(s["cache"], s["read"], c["dim"], s["q"].dtype))
    if op == "tree4":
        return gb.tree_attention_int4(s["q"], s["cache"], s["table"], s["lens"], page_size=c["page"],
                                      next_n=c["next_n"], tree_mask=s["mask"], return_lse=True)
    if op == "selected4":
        return gb.selected_attention_int4(s["q"], s["cache"], s["idx"], return_lse=True)
    return gb.prompt_attention(s["q"], s["k"], s["v"], s["cu"], cu_seqlens_k=s["cu_k"] if c["context"] else None,
                               out=s["out"], lse=s["lse"])


# --------------------------------------------------------------------- work

def work(case):
    op, d, kv, qh = case["op"], case["dim"], case["kv_heads"], case["q_heads"]
    if op in ("rotate", "quantise"):
        n = case["tokens"]
        moved = n * (4 * qh * d + 4 * kv * d + 8)
        moved += n * 4 * kv * d if op == "rotate" else n * kv * d * 9 / 8
        back = (n + case["context"]) * kv * d * (9 / 8 + 4) if op == "quantise" else 0
        return {"bytes": moved + back, "flops": n * (qh + kv) * d * 8 + back}
    if op == "prompt":
        mean = case["len_max"] if case["batch"] == 1 else (case["len_min"] + case["len_max"]) / 2
        square = mean * mean if case["batch"] == 1 else (case["len_min"] ** 2 + case["len_min"] * case["len_max"] + case["len_max"] ** 2) / 3
        context = 0.75 * case["context"]
        idle = 1 - 1 / case["batch"] if case["batch"] >= 8 else 1
        pairs = case["batch"] * idle * ((square + mean) / 2 + mean * context)
        return {"bytes": case["batch"] * idle * (mean * qh * (4 * d + 4) + (mean + context) * 4 * kv * d),
                "flops": 4 * pairs * qh * d}
    if op == "selected4":
        pairs = case["rows"] * case["top_k"] * (1 - case["short"] / 2)
        return {"bytes": pairs * (kv * d * 9 / 8 + 4) + case["rows"] * qh * (4 * d + 4), "flops": 4 * pairs * qh * d}
    mean = case["len_max"] if case["batch"] == 1 else (case["len_min"] + case["len_max"]) / 2
    tokens = mean * case["batch"]
    rows = case["batch"] * case["next_n"] * qh
    return {"bytes": tokens * kv * d * 9 / 8 + rows * (4 * d + 4), "flops": 4 * rows * mean * d}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in 64 bits, request by request."""
    def decode(rows):
        """Byte tables: each code byte holds bits of two neighbouring pairs."""
        d = case["dim"]
        c, w = 16 * ((d + 31) // 32), 8 if d <= 128 else 16
        out = []
        for part in (0, 1):
            raw = rows[:, part * c:part * c + d // 2].long().view(rows.shape[0], d // 8, 4)
            word = raw[..., 0] + raw[..., 1] * 256 + raw[..., 2] * 65536 + raw[..., 3] * 16777216
            x = torch.zeros((rows.shape[0], d // 8, 8), dtype=torch.float64, device=rows.device)
            for j in range(4):
                turned = (word >> 4 * j) | ((word << (32 - 4 * j)) & 0xffffffff)
                low, high = turned & 0xffff, turned >> 16
                x[..., 2 * j] = (1 - 2 * (low >> 15)).double() * (low & 7)
                x[..., 2 * j + 1] = (1 - 2 * (high >> 15 & 1)).double() * (high & 7)
            byte = rows[:, 2 * c + part * w:2 * c + part * w + d // 16].long() % 128
            scale = torch.tensor([b / 512 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 10) for b in range(128)],
                                 dtype=torch.float64, device=rows.device)[byte]
            out.append((x.view(rows.shape[0], d // 16, 16) * scale.unsqueeze(2)).view(rows.shape[0], d))
        return out

    def attend(q, k, v, see):
        """Rows [t, group, dim] over keys [n, dim], see [t, n]."""
        x = torch.einsum("tgd,nd->tgn", q.double(), k) * case["dim"] ** -0.5
        x = x.masked_fill(~see.unsqueeze(1), -math.inf)
        lse = torch.logsumexp(x, 2) if k.shape[0] else torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
        p = torch.where(lse.unsqueeze(2) == -math.inf, 0.0, (x - lse.unsqueeze(2)).exp())
        return torch.einsum("tgn,nd->tgd", p, v), lse

    def heads(s, rows, out, lse, kv_of, see):
        g = case["q_heads"] // case["kv_heads"]
        for h in range(case["kv_heads"]):
            k, v = kv_of(h)
            out[rows, h * g:h * g + g], lse[rows, h * g:h * g + g] = attend(s["q"][rows, h * g:h * g + g], k, v, see)

    def empty(s):
        return torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device), \
            torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)

    def turn(x, w, s):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(2, keepdim=True) / case["dim"] + 1e-6).sqrt() * w.double()
        y, half = x.clone(), case["rotary"] // 2
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            angle = (s["positions"].double() * float(s["freq"][i])).unsqueeze(1)
            y[:, :, a] = x[:, :, a] * angle.cos() - x[:, :, b] * angle.sin()
            y[:, :, b] = x[:, :, a] * angle.sin() + x[:, :, b] * angle.cos()
        return y

    def coded(x):
        """What the 4-bit codes of [..., dim] stand for."""
        n = x.shape[-1] // 16
        x = x.double().reshape(x.shape[:-1] + (n, 16))
        a = torch.true_divide(x.abs().max(-1, keepdim=True).values, torch.full_like(x[..., :1], 7))
        _, e = torch.frexp(a)
        powers = torch.tensor([2.0 ** (i - 9) for i in range(40)], dtype=torch.float64, device=x.device)
        step = powers[(e - 4).clamp(min=-9, max=30).long() + 9]      # of 4 significant bits
        scale = ((a / step).round() * step).clamp(max=448)
        y = torch.where(scale == 0, 0.0, (x / scale).round().clamp(-7, 7) * scale)
        return y.reshape(y.shape[:-2] + (n * 16,))

    def rotate(s):
        out = [turn(s["q"], s["wq"], s), s["k_cache"].double(), s["v_cache"].double()]
        k = turn(s["k"], s["wk"], s)
        live = [i for i, x in enumerate(s["slots"].tolist()) if x >= 0]
        to = s["slots"][live].long()
        out[1][to], out[2][to] = k[live], s["v"][live].double()
        return tuple(out)

    def quantise(s):
        rows = s["cache"].shape[0]
        k, v = zip(*(decode(s["cache"][:, h]) for h in range(case["kv_heads"])))
        k, v = torch.stack(k, 1), torch.stack(v, 1)
        live = [i for i, x in enumerate(s["slots"].tolist()) if x >= 0]
        to = s["slots"][live].long()
        k[to], v[to] = coded(turn(s["k"], s["wk"], s))[live], coded(s["v"])[live]
        assert k.shape[0] == rows
        return turn(s["q"], s["wq"], s), k[s["read"].long()], v[s["read"].long()]

    def tree4(s):
        out, lse = empty(s)
        n = case["next_n"]
        for i in range(case["batch"]):
            length = int(s["lens"][i])
            pages = s["table"][i].long()
            at = torch.arange(length, device=pages.device)
            slots = pages[at // case["page"]] * case["page"] + at % case["page"]
            see = torch.ones((n, length), dtype=torch.bool)
            for t in range(n):
                bits = int(s["tree"][i * n + t]) & ((1 << 64) - 1)
                for j in range(n):
                    if 0 <= length - n + j:
                        see[t, length - n + j] = bool(bits >> j & 1)
            heads(s, slice(i * n, i * n + n), out, lse, lambda h: decode(s["cache"][slots, h]), see.to(pages.device))
        return out, lse

    def selected4(s):
        out, lse = empty(s)
        for r in range(case["rows"]):
            slots = s["idx"][r][s["idx"][r] >= 0].long()
            see = torch.ones((1, slots.numel()), dtype=torch.bool, device=slots.device)
            heads(s, slice(r, r + 1), out, lse, lambda h: decode(s["cache"][slots, h]), see)
        return out, lse

    def prompt(s):
        out, lse = empty(s)
        cu, cu_k = s["cu"].tolist(), s["cu_k"].tolist()
        for i in range(case["batch"]):
            n = cu_k[i + 1] - cu_k[i]
            # some thousand rows at a time
            for t0 in range(cu[i], cu[i + 1], 2048):
                t1 = min(t0 + 2048, cu[i + 1])
                last = torch.arange(t0, t1, device=out.device) - cu[i + 1] + n
                see = torch.arange(n, device=out.device) <= last.unsqueeze(1)
                heads(s, slice(t0, t1), out, lse,
                      lambda h: [s[x][cu_k[i]:cu_k[i] + n, h].double() for x in "kv"], see)
        return out, lse

    pairs = work(case)["flops"]
    if pairs > 4e12:
        return None
    return {"rotate": rotate, "quantise": quantise, "tree4": tree4, "selected4": selected4,
            "prompt": prompt}[case["op"]](prepare(case, seed))
