"""Attention over 4-bit caches on the GPU against its definition in 64 bits.

Tolerances, fixed beforehand, as for the 16-bit caches: u |out| for the output's
own rounding, and (w + 2 eta) sum p |v| with eta the bound on a score's error
and w what a probability is rounded by: 2^-8 in bf16; in fp16 it is the sum of
two bf16 numbers, 2^-16.  lse by eta and 32-bit rounding.  A probability below
2^-126 of its row's reference is 0 in 32 bits: the reference is no larger than
the largest score, so the sum is at least 1 and the output misses at most
2^-126 of each value."""
import math

import numpy as np
import pytest
import torch

import decode_reference as dref
import prefill_reference as ref
import sparse_attention_top_gb300 as gb

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
W = {BF: 2.0 ** -8, HF: 2.0 ** -16}
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def trees(requests, n, seed, empty=False):
    r = np.random.RandomState(seed)
    rows = np.zeros((requests, n), dtype=np.uint64)
    for i in range(requests):
        rows[i, 0] = 1
        for k in range(1, n):
            rows[i, k] = rows[i, r.randint(max(0, k - 4), k)] | (np.uint64(1) << np.uint64(k))
        if empty:
            rows[i, 0] = 0
    return rows.reshape(-1).view(np.int64).copy()


class Batch:
    """A paged 4-bit batch on the CPU; rows that no request owns are random
    bytes, the largest scales among them."""

    def __init__(self, lens, next_n, q_heads, kv, dim, page, dtype, seed, cols=None, head_major=False, size=None,
                 ordered=False):
        g = torch.Generator().manual_seed(seed)
        b = len(lens)
        cols = max(1, -(-max(max(lens), 1) // page)) if cols is None else cols
        pages = b * cols + 2
        self.table = torch.randperm(pages, generator=g).to(torch.int32)[:b * cols].view(b, cols).clone()
        if ordered:      # positions in the slots' order
            self.table = torch.arange(b * cols, dtype=torch.int32).view(b, cols)
        slots = pages * page
        k, v = torch.randn((2, slots, kv, dim), generator=g)
        if size is not None:
            k = k * size(slots, g)
        rows = ref.row_bytes(*ref.codes(k.numpy()), *ref.codes(v.numpy()))
        used = np.zeros(slots, dtype=bool)
        for i, n in enumerate(lens):
            for p in range(max(0, min(n, cols * page))):
                used[int(self.table[i, p // page]) * page + p % page] = True
        junk = torch.randint(0, 256, rows.shape, generator=g, dtype=torch.uint8).numpy()
        rows[~used] = junk[~used]
        self.rows, self.dim, self.head_major = rows, dim, head_major
        self.q = torch.randn((b * next_n, q_heads, dim), generator=g).to(dtype)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.page, self.next_n, self.group, self.dtype = page, next_n, q_heads // kv, dtype
        self.scale = dim ** -0.5

    def cache(self, dev):
        t = torch.from_numpy(self.rows)
        if self.head_major:
            return t.transpose(0, 1).contiguous().to(dev).transpose(0, 1)
        return t.to(dev)


def check_rows(b, out, lse, seen_of, scale=None, units=(1.0, 1.0)):
    k, v = ref.values(b.rows, b.dim)
    k, v = k * units[0], v * units[1]
    q = b.q.double().numpy()
    scale = b.scale if scale is None else scale
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    small = 2.0 ** -25 if b.dtype is HF else 0.0
    for r in range(q.shape[0]):
        o, l, eta, mag = dref.attend(q[r], k if scale >= 0 else -k, v, seen_of(r), b.group, abs(scale))
        none = l == -math.inf
        assert np.array_equal(none, lse[r] == -math.inf)
        tol = U[b.dtype] * np.abs(o) + (W[b.dtype] + 2 * eta[:, None]) * mag + small
        tol = tol + 2.0 ** -126 * len(seen_of(r)) * np.abs(v).max()
        bad = np.abs(out[r] - o) > tol
        assert not bad.any(), (r, np.argwhere(bad)[:5], np.max(np.abs(out[r] - o) - tol))
        at = ~none
        assert np.all(np.abs(lse[r][at] - l[at]) <= eta[at] + 2.0 ** -21 * (1 + np.abs(l[at])))


def check_tree(dev, b, tree=None, units=(1.0, 1.0), **kw):
    cache = b.cache(dev)
    mask = None if tree is None else torch.from_numpy(tree).to(dev)
    out, lse = gb.tree_attention_int4(b.q.to(dev), cache, b.table.to(dev), b.lens.to(dev), page_size=b.page, next_n=b.next_n,
                                      tree_mask=mask, return_lse=True, k_scale=units[0], v_scale=units[1], **kw)
    torch.cuda.synchronize(dev)
    table, lens, slots = b.table.numpy(), b.lens.numpy(), cache.shape[0]
    check_rows(b, out, lse, lambda r: dref.visible(table, b.page, slots, lens, b.next_n, tree, r), kw.get("scale"), units)
    return out, lse


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,next_n,q_heads,kv,dim,page,tree", [
    ([1], 1, 1, 1, 64, 1, False),                        # one token over itself
    ([130, 0, 1, 127, 128, 129, 300], 1, 8, 2, 128, 16, False),
    ([5, 2, 0, 3, 257], 4, 4, 4, 64, 7, False),          # shorter than its drafts
    ([400, 64, 65, 20], 64, 2, 1, 128, 64, True),        # 128 rows a head: two row tiles, the mask's last bit
    ([260, 140], 33, 16, 2, 96, 100, True),              # 264 rows a head: a row tile of eight
    ([333], 5, 7, 7, 16, 32, True),                      # the smallest head
    ([200, 190], 3, 12, 2, 256, 128, True),              # the largest: 18 rows
    ([300, 7], 8, 12, 2, 208, 16, True),                 # 48 rows above dimension 128: two row tiles
    ([150], 2, 6, 1, 80, 1, False),
    ([700, 41], 16, 32, 2, 112, 48, True),
    ([513, 700], 4, 32, 4, 128, 64, False),              # 32 rows
    ([900], 17, 1, 1, 48, 3, True),
])
def test_tree_attention_int4(dev, dtype, lens, next_n, q_heads, kv, dim, page, tree):
    b = Batch(lens, next_n, q_heads, kv, dim, page, dtype, seed=len(lens) * 31 + dim, head_major=dim in (128, 256))
    check_tree(dev, b, trees(len(lens), next_n, 5) if tree else None)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_empty_rows_missing_pages(dev, dtype):
    """Rows whose mask leaves nothing, negative and foreign pages, lengths beyond the table."""
    b = Batch([300, 260, 9000, 3, -4], 3, 8, 2, 64, 32, dtype, seed=3, cols=10)
    b.table[0, 2], b.table[1, 0], b.table[2, 9] = -1, 1 << 29, -7
    tree = trees(5, 3, 8, empty=True)
    tree[9:12] = 0                       # all rows of request 3
    out, lse = check_tree(dev, b, tree)
    assert bool((out[9:] == 0).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("scale,units", [(-0.125, (1.0, 1.0)), (0.0, (1.0, 1.0)), (3.0, (0.25, 64.0)), (None, (2.0 ** -20, 2.0 ** 20))])
def test_scales(dev, dtype, scale, units):
    b = Batch([700, 64], 2, 8, 2, 128, 16, dtype, seed=4)
    if units[1] > 2.0 ** 10 and dtype is HF:
        units = (units[0], 2.0 ** -6)    # (within fp16's range)
    check_tree(dev, b, scale=scale, units=units) if scale is not None else check_tree(dev, b, units=units)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["rising", "sink", "jumps"])
@pytest.mark.parametrize("q_heads,next_n", [(4, 1), (32, 1), (12, 8)])
@pytest.mark.parametrize("junk", [False, True])
def test_references_move(dev, dtype, kind, q_heads, next_n, junk):
    """Scores that grow along the context, one key far above the others, and
    tiles that jump: every row's reference moves many times."""
    def size(slots, g):
        at = torch.arange(slots).view(-1, 1, 1)
        if kind == "rising":
            return 0.2 + at / 60.0
        if kind == "sink":
            return torch.where(at % 611 == 7, 40.0, 0.5)
        return torch.exp(3 * torch.randn((slots, 1, 1), generator=g))
    b = Batch([1500, 611], next_n, q_heads, 1, 64, 64, dtype, seed=9, size=size, ordered=not junk)
    b.table = torch.arange(b.table.numel(), dtype=torch.int32).view(b.table.shape)   # (rows of random bytes among them)
    check_tree(dev, b)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("batch,length,next_n,q_heads,kv,dim", [
    (1, 40000, 2, 2, 1, 64),          # one unit over all blocks
    (40, 700, 1, 16, 8, 128),         # several units a block
    (3, 9000, 8, 16, 2, 128),         # 64 rows, split
    (2, 6000, 1, 8, 2, 256),
])
def test_many_tiles(dev, dtype, batch, length, next_n, q_heads, kv, dim):
    lens = [length - 37 * i % 500 for i in range(batch)]
    b = Batch(lens, next_n, q_heads, kv, dim, 64, dtype, seed=length)
    first = check_tree(dev, b)
    again = gb.tree_attention_int4(b.q.to(dev), b.cache(dev), b.table.to(dev), b.lens.to(dev), page_size=64, next_n=next_n,
                                   return_lse=True)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows,top_k,q_heads,kv,dim", [
    (1, 0, 2, 1, 64), (3, 1, 4, 4, 16), (7, 130, 8, 2, 128), (64, 300, 16, 1, 96), (5, 257, 40, 1, 128), (3, 200, 2, 2, 256)])
def test_selected_attention_int4(dev, dtype, rows, top_k, q_heads, kv, dim):
    b = Batch([600], 1, q_heads, kv, dim, 1, dtype, seed=rows + top_k)
    g = torch.Generator().manual_seed(top_k)
    n = b.rows.shape[0]
    idx = torch.randint(-50, n + 9, (rows, top_k), generator=g, dtype=torch.int32)     # absent and foreign entries among them
    if rows > 2:
        idx[1] = -1                                                                    # a row without any
        idx[2] = idx[2, :1]                                                            # one slot, listed over and over
    b.q = torch.randn((rows, q_heads, dim), generator=g).to(dtype)
    wide = torch.full((rows, top_k + 3), -1, dtype=torch.int32)
    wide[:, :top_k] = idx
    out, lse = gb.selected_attention_int4(b.q.to(dev), b.cache(dev), wide.to(dev)[:, :top_k], return_lse=True)
    check_rows(b, out, lse, lambda r: dref.selected(idx.numpy(), n, r))


def test_query_values(dev):
    """An infinite or NaN query row stays with itself; fp16 queries at the ends of their range."""
    b = Batch([300], 3, 2, 1, 64, 16, HF, seed=2)
    b.q[0, 0, 3], b.q[1, 1, 5] = math.inf, math.nan
    b.q[2, 0] = torch.linspace(-6.0e4, 6.0e4, 64).to(HF)
    b.q[2, 1] = torch.arange(64).to(HF) * 2.0 ** -24
    out, lse = gb.tree_attention_int4(b.q.to(dev), b.cache(dev), b.table.to(dev), b.lens.to(dev), page_size=16, next_n=3,
                                      return_lse=True)
    assert bool(torch.isfinite(out[0, 1]).all() and torch.isfinite(out[1, 0]).all() and torch.isfinite(out[2]).all())
    assert bool(torch.isnan(out[1, 1]).all())
    b.q[0, 0, 3], b.q[1, 1, 5] = 0.0, 0.0
    b.q[0], b.q[1] = 1.0, 1.0
    out[0], out[1] = 0, 0
    seen = dref.visible(b.table.numpy(), 16, b.rows.shape[0], b.lens.numpy(), 3, None, 2)
    k, v = ref.values(b.rows, 64)
    o, l, eta, mag = dref.attend(b.q[2].double().numpy(), k, v, seen, 2, b.scale)
    assert np.all(np.abs(out[2].cpu().double().numpy() - o) <= U[HF] * np.abs(o) + (W[HF] + 2 * eta[:, None]) * mag + 2.0 ** -25)


def test_replays_other_lengths(dev):
    """A captured call follows the lengths, pages and cache of its replay."""
    b = Batch([900, 300, 20], 2, 8, 2, 128, 16, BF, seed=6)
    q, cache, table, lens = b.q.to(dev), b.cache(dev), b.table.to(dev), b.lens.to(dev)
    own = torch.zeros(gb.gbtopk_attention_workspace_bytes(6, 8, 2, 128), dtype=torch.uint8, device=dev)
    call = lambda: gb.tree_attention_int4(q, cache, table, lens, page_size=16, next_n=2, return_lse=True, workspace=own)  # noqa: E731
    call()
    torch.cuda.synchronize(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for new in ([1, 0, 900], [899, 2, 450]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize(dev)
        kept = [x.clone() for x in got]
        b.lens = torch.tensor(new, dtype=torch.int32)
        check_rows(b, *kept, lambda r: dref.visible(b.table.numpy(), 16, b.rows.shape[0], b.lens.numpy(), 2, None, r))


def test_far_slots(dev):
    """Rows beyond 2^31 bytes into the cache."""
    dim, kv = 128, 8
    n = gb.int4_row_bytes(dim)
    slots = (1 << 31) // (n * kv) + 70000
    cache = torch.zeros((slots, kv, n), dtype=torch.uint8, device=dev)
    b = Batch([500], 1, 8, 8, dim, 1, BF, seed=5)
    at = torch.arange(500, dtype=torch.int32) * 137 + (slots - 69000)
    rows = b.rows[b.table[0].numpy()[:500]]
    cache[at.long().to(dev)] = torch.from_numpy(rows).to(dev)
    out, lse = gb.selected_attention_int4(b.q.to(dev), cache, at.view(1, -1).to(dev), return_lse=True)
    b.rows = rows
    check_rows(b, out, lse, lambda r: [(j, j) for j in range(500)])
    k, v = gb.read_cache_int4(cache, at.to(dev), dim, HF)
    a, c = ref.values(rows, dim)
    assert torch.equal(k.cpu(), torch.from_numpy(a).to(HF)) and torch.equal(v.cpu(), torch.from_numpy(c).to(HF))


def test_attention_int4_refuses(dev):
    b = Batch([100], 2, 4, 2, 64, 16, BF, seed=1)
    q, cache, table, lens = b.q.to(dev), b.cache(dev), b.table.to(dev), b.lens.to(dev)

    def tree(**kw):
        a = dict(q=q, cache=cache, page_table=table, seq_lens=lens, page_size=16, next_n=2)
        a.update(kw)
        return gb.tree_attention_int4(**a)

    def selected(**kw):
        a = dict(q=q, cache=cache, indices=table.repeat(2, 1))
        a.update(kw)
        return gb.selected_attention_int4(**a)

    tree(), selected()
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(cache=cache.to(torch.int8)), dict(cache=cache[..., :64]),
                dict(cache=cache[:, :, ::2]), dict(k_scale=0.0), dict(v_scale=1.5), dict(out=q.float()), dict(lse=torch.zeros(2, device=dev)),
                dict(workspace=torch.zeros(64, dtype=torch.uint8, device=dev)), dict(q=q.cpu()), dict(cache=cache.cpu())):
        for f in (tree, selected):
            with pytest.raises(ValueError):
                f(**bad)
    for bad in (dict(next_n=3), dict(next_n=0), dict(page_size=0), dict(seq_lens=lens.long()), dict(page_table=table.long()),
                dict(tree_mask=lens), dict(page_table=table.expand(2, -1))):
        with pytest.raises(ValueError):
            tree(**bad)
    with pytest.raises(ValueError):
        selected(indices=table)
