"""The decode-step operators in 64 bits, one request, row and head at a time.

Plain restatements of the definitions in include/gbtopk.h, for the tests:
loops over Python numbers and float64 arrays, nothing of the package.  Each
returns, beside the result, what bounds a kernel's error."""
import math

import numpy as np

U = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}     # unit roundoff of the 16-bit types


def bits_of(x):
    return int(x) & ((1 << 64) - 1)


def slot_of(table_row, page_size, num_slots, p):
    c = p // page_size
    if p < 0 or c >= len(table_row) or table_row[c] < 0:
        return -1
    s = int(table_row[c]) * page_size + p % page_size
    return s if s < num_slots else -1


def visible(table, page_size, num_slots, lens, next_n, tree, r):
    """(position, slot) pairs that row r sees."""
    i, t = divmod(r, next_n)
    length = int(lens[i])
    ctx = length - next_n
    mask = bits_of(tree[r]) if tree is not None else (1 << (t + 1)) - 1
    seen = []
    for p in range(max(0, min(length, table.shape[1] * page_size))):
        if p >= ctx and not mask >> (p - ctx) & 1:
            continue
        s = slot_of(table[i], page_size, num_slots, p)
        if s >= 0:
            seen.append((p, s))
    return seen


def selected(indices, num_slots, r):
    return [(j, int(s)) for j, s in enumerate(indices[r]) if 0 <= s < num_slots]


def attend(q, k, v, seen, group, scale):
    """One row [heads, dim] over its (position, slot) list.  Returns out,
    lse, and per head: eta, a bound on the error of a score computed with a
    32-bit running sum (which may truncate: dim * 2^-23 of the sum of
    magnitudes, and of the score's own rounding), and sum p |v|."""
    heads, dim = q.shape
    out, mag = np.zeros((heads, dim)), np.zeros((heads, dim))
    lse, eta = np.full(heads, -math.inf), np.zeros(heads)
    if not seen:
        return out, lse, eta, mag
    slots = [s for _, s in seen]
    for h in range(heads):
        kk, vv = k[slots, h // group], v[slots, h // group]
        s = scale * (kk @ q[h])
        top = s.max()
        lse[h] = top + math.log(np.exp(s - top).sum())
        p = np.exp(s - lse[h])
        out[h], mag[h] = p @ vv, p @ np.abs(vv)
        eta[h] = (dim + 8) * 2.0 ** -23 * (scale * (np.abs(kk) @ np.abs(q[h]))).max() + 2.0 ** -20
    return out, lse, eta, mag


def weights(q, k, lse, w, table, page_size, num_slots, lens, next_n, tree, accept, group, scale):
    """The updated weights and, per entry, the error allowed: exp's argument
    error on every term, the running sum's rounding, the final addition's."""
    w = w.astype(np.float64).copy()
    tol = np.abs(w) * 2.0 ** -23
    heads, dim = q.shape[1:]
    for r in range(q.shape[0]):
        i, t = divmod(r, next_n)
        if accept is not None and not bits_of(accept[i]) >> t & 1:
            continue
        for p, s in visible(table, page_size, num_slots, lens, next_n, tree, r):
            if p >= w.shape[2]:
                continue
            for h in range(heads):
                if lse[r, h] == -math.inf:
                    continue
                x = scale * (k[s, h // group] @ q[r, h])
                eta = (dim + 8) * 2.0 ** -23 * scale * (np.abs(k[s, h // group]) @ np.abs(q[r, h])) + 2.0 ** -20
                add = math.exp(x - float(lse[r, h]))
                at = (i, 0 if w.shape[1] == 1 else h // group, p)
                w[at] += add
                tol[at] += add * (1.5 * eta + abs(float(lse[r, h])) * 2.0 ** -22 + heads * next_n * 2.0 ** -23)
    return w, tol


def evict(w, lens, table, page_size, next_n, accept, budget, recent):
    """Kept positions of each (request, weight head), ascending."""
    kept = []
    for i in range(w.shape[0]):
        length = int(lens[i])
        alive = list(range(max(0, min(length, table.shape[1] * page_size, w.shape[2]))))
        if accept is not None:
            bits = bits_of(accept[i])
            alive = [p for p in alive if p < length - next_n or bits >> (p - length + next_n) & 1]
        rows = []
        for h in range(w.shape[1]):
            if len(alive) <= budget:
                rows.append(alive)
                continue
            last = min(recent, budget)
            cut = len(alive) - last
            best = sorted(alive[:cut], key=lambda p: (-float(w[i, h, p]), p))[:budget - last]
            rows.append(sorted(best) + alive[cut:])
        kept.append(rows)
    return kept


def verify(logits, tokens, uniforms, noise, next_n, tree=None, temperature=None, draft=None):
    """One tuple (accepted, path, next token, mask) a request."""
    got = []
    vocab = logits.shape[1]
    for i in range(logits.shape[0] // next_n):
        temp = 1.0 if temperature is None else float(temperature[i])
        parent = {}
        for n in range(1, next_n):
            above = [a for a in range(n) if tree is None and a == n - 1 or
                     tree is not None and bits_of(tree[i * next_n + n]) >> a & 1]
            if above:
                parent[n] = max(above)
        cur, path = 0, [0]
        while True:
            x = logits[i * next_n + cur].astype(np.float64)
            top = x.max()
            if top == -math.inf:
                rest = np.zeros(vocab)
            elif temp > 0:
                rest = np.exp((x - top) / temp)
                rest /= rest.sum()
            else:
                rest = np.zeros(vocab)
                rest[int(np.argmax(x))] = 1.0
            mass, nxt = 1.0, None
            for n in range(cur + 1, next_n):
                if parent.get(n) != cur:
                    continue
                tok, u = int(tokens[i * next_n + n]), float(uniforms[i * next_n + n])
                ok = 0 <= tok < vocab
                have = rest[tok] if ok else 0.0
                if draft is not None:
                    q = draft[i * next_n + cur].astype(np.float64)
                    if u * (q[tok] if ok else 1.0) < have:
                        nxt = n
                        break
                    rest = np.maximum(rest - q, 0.0)
                else:
                    if u * mass < have:
                        nxt = n
                        break
                    mass -= have
                    if ok:
                        rest[tok] = 0.0
            if nxt is None:
                break
            cur = nxt
            path.append(cur)
        race = np.where(rest > 0, rest / noise[i].astype(np.float64), 0.0)
        follow = int(np.argmax(race)) if race.max() > 0 else -1
        got.append((len(path) - 1, path + [-1] * (next_n - len(path)), follow, sum(1 << n for n in path)))
    return got
