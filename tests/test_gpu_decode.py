"""The decode-step operators on the GPU against their definitions in 64 bits.

Tolerances come from the arithmetic and are fixed beforehand: with u the unit
roundoff of the 16-bit type and eta the bound on a score's error (32-bit sums),
an attention output may be off by u |out| (its own rounding) plus (u + 2 eta)
sum p |v| (probabilities rounded to the type, scores off by eta); lse by eta
and 32-bit rounding.  Kept positions, moved rows, accepted paths and drawn
tokens are exact."""
import math

import numpy as np
import pytest
import torch

import decode_reference as ref
import sparse_attention_top_gb300 as gb

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def trees(requests, n, seed, empty=False):
    """Ancestor bits of random trees; with ``empty``, node 0's row sees nothing."""
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
    """A paged batch on the CPU: pages in random order, everything that no
    request owns poisoned with NaN."""

    def __init__(self, lens, next_n, q_heads, kv_heads, dim, page, dtype, seed, cols=None, fused=False, spare=0):
        g = torch.Generator().manual_seed(seed)
        b = len(lens)
        cols = max(1, -(-max(max(lens), 1) // page)) if cols is None else cols
        more = -(-spare // page)
        pages = b * (cols + more) + 2
        order = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = order[:b * cols].view(b, cols).clone()
        self.new_table = order[b * cols:b * (cols + more)].view(b, more).clone()
        shape = (pages * page, 2, kv_heads, dim) if fused else (2, pages * page, kv_heads, dim)
        kv = torch.randn(shape, generator=g).to(dtype)
        used = torch.zeros(pages * page, dtype=torch.bool)
        for i, n in enumerate(lens):
            for p in range(max(0, min(n, cols * page))):
                used[int(self.table[i, p // page]) * page + p % page] = True
        k, v = (kv[:, 0], kv[:, 1]) if fused else (kv[0], kv[1])
        k[~used] = math.nan
        v[~used] = math.nan
        self.kv, self.fused = kv, fused
        self.q = torch.randn((b * next_n, q_heads, dim), generator=g).to(dtype)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.page, self.next_n, self.group = page, next_n, q_heads // kv_heads
        self.scale = dim ** -0.5
        self.u = ref.U[str(dtype).replace("torch.", "")]

    def caches(self, dev):
        kv = self.kv.to(dev)
        return (kv[:, 0], kv[:, 1]) if self.fused else (kv[0], kv[1])

    def wide(self):
        k, v = (self.kv[:, 0], self.kv[:, 1]) if self.fused else (self.kv[0], self.kv[1])
        return self.q.double().numpy(), k.double().numpy(), v.double().numpy()


def check_rows(b, out, lse, seen_of):
    q, k, v = b.wide()
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    for r in range(q.shape[0]):
        o, l, eta, mag = ref.attend(q[r], k, v, seen_of(r), b.group, b.scale)
        none = l == -math.inf
        assert np.array_equal(none, lse[r] == -math.inf)
        tol = b.u * np.abs(o) + (b.u + 2 * eta[:, None]) * mag
        assert np.all(np.abs(out[r] - o) <= tol), (r, np.max(np.abs(out[r] - o) - tol))
        at = ~none
        assert np.all(np.abs(lse[r][at] - l[at]) <= eta[at] + 2.0 ** -21 * (1 + np.abs(l[at])))


def check_tree(dev, b, tree=None, **kw):
    k, v = b.caches(dev)
    mask = None if tree is None else torch.from_numpy(tree).to(dev)
    out, lse = gb.tree_attention(b.q.to(dev), k, v, b.table.to(dev), b.lens.to(dev), page_size=b.page,
                                 next_n=b.next_n, tree_mask=mask, return_lse=True, **kw)
    torch.cuda.synchronize(dev)
    table, lens, slots = b.table.numpy(), b.lens.numpy(), k.shape[0]
    check_rows(b, out, lse, lambda r: ref.visible(table, b.page, slots, lens, b.next_n, tree, r))
    return out, lse


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,next_n,q_heads,kv_heads,dim,page,tree", [
    ([1], 1, 1, 1, 64, 1, False),                        # one token over itself
    ([130, 0, 1, 127, 128, 129, 300], 1, 8, 2, 128, 16, False),
    ([5, 2, 0, 3, 257], 4, 4, 4, 64, 7, False),          # shorter than its drafts
    ([400, 64, 65, 20], 64, 2, 1, 128, 64, True),        # 128 rows a head, the mask's last bit
    ([260, 140], 33, 16, 2, 96, 100, True),              # 264 rows a head: several row tiles
    ([333], 5, 7, 7, 8, 32, True),                       # the smallest head
    ([200, 190], 3, 12, 2, 256, 128, True),              # the largest
    ([150], 2, 6, 1, 80, 1, False),
    ([700, 41], 16, 32, 2, 72, 48, True),                # 256 rows a head
])
def test_tree_attention(dev, dtype, lens, next_n, q_heads, kv_heads, dim, page, tree):
    b = Batch(lens, next_n, q_heads, kv_heads, dim, page, dtype, seed=len(lens) * 31 + dim, fused=dim == 128)
    check_tree(dev, b, trees(len(lens), next_n, 5) if tree else None)


def test_tree_attention_rows_that_see_nothing(dev):
    """No context and an empty mask: zeros and -inf beside ordinary rows; a
    draft that no row sees may hold anything."""
    b = Batch([4, 4, 9], 4, 4, 2, 64, 4, BF, seed=3)
    tree = trees(3, 4, 7, empty=True)
    unseen = np.uint64(~(1 << 3) & ((1 << 64) - 1))
    tree = (tree.view(np.uint64) & unseen).view(np.int64).copy()
    for i in range(3):
        p = int(b.lens[i]) - 1
        s = int(b.table[i, p // 4]) * 4 + p % 4
        b.kv[:, s] = math.inf if i else math.nan
    out, lse = check_tree(dev, b, tree)
    assert not out[0].any() and not out[4].any()
    assert torch.isinf(lse[0]).all() and torch.isfinite(lse[8]).all()


def test_tree_attention_pages_that_do_not_exist(dev):
    """Negative and too large page ids, and lengths beyond the table."""
    b = Batch([100, 90, 64], 2, 4, 1, 64, 16, HF, seed=11)
    b.table[0, 2] = -1
    b.table[1, 0] = 1 << 20
    b.table[1, 1] = 2 ** 31 - 1
    b.table[2, :] = -5
    b.lens = torch.tensor([5000, 90, 64], dtype=torch.int32)
    for i, n in ((0, 112),):
        for p in range(n):
            s = ref.slot_of(b.table[i].numpy(), 16, b.kv.shape[1], p)
            if s >= 0:
                b.kv[:, s] = torch.nan_to_num(b.kv[:, s], nan=0.5)
    check_tree(dev, b)


def test_tree_attention_negative_lengths_are_empty(dev):
    b = Batch([40, 1], 2, 4, 2, 64, 8, BF, seed=2)
    b.lens = torch.tensor([-2 ** 31, -1], dtype=torch.int32)
    out, lse = check_tree(dev, b)
    assert not out.any() and torch.isinf(lse).all()


def test_tree_attention_scale_and_large_scores(dev):
    """Scores over a wide range: the running maximum moves, exp underflows."""
    b = Batch([600, 390], 3, 8, 2, 64, 32, BF, seed=23)
    b.q *= 8
    b.scale = 0.5
    check_tree(dev, b, scale=0.5)


def test_tree_attention_strides_and_caller_buffers(dev):
    b = Batch([77, 260], 2, 8, 4, 64, 16, HF, seed=9)
    k, v = b.caches(dev)
    wide = torch.full((b.q.shape[0], 8, 96), math.nan, dtype=HF, device=dev)
    wide[:, :, :64] = b.q.to(dev)
    padded = torch.full((2, b.table.shape[1] + 5), -9, dtype=torch.int32, device=dev)
    padded[:, :b.table.shape[1]] = b.table.to(dev)
    out = torch.full((4 + 2, 8, 64), 7.0, dtype=HF, device=dev)
    lse = torch.full((4 + 2, 8), 7.0, device=dev)
    ws = torch.zeros(gb.gbtopk_attention_workspace_bytes(4, 8, 4, 64), dtype=torch.uint8, device=dev)
    ws[256:] = 255
    got = gb.tree_attention(wide[:, :, :64], k, v, padded[:, :b.table.shape[1]], b.lens.to(dev), page_size=16, next_n=2,
                            out=out[1:5], lse=lse[1:5], workspace=ws)
    torch.cuda.synchronize(dev)
    assert got[0].data_ptr() == out[1:5].data_ptr()
    table, lens = b.table.numpy(), b.lens.numpy()
    check_rows(b, out[1:5], lse[1:5], lambda r: ref.visible(table, 16, k.shape[0], lens, 2, None, r))
    for t in (out, lse):    # the rows around stay as they were
        assert (t[0] == 7).all() and (t[5] == 7).all()
    assert gb.gbtopk_device_status(ws) == 0


def test_tree_attention_offsets_beyond_32_bits(dev):
    """Slots whose element offset passes 2^32."""
    slots, heads, dim = (1 << 32) // 1024 + 4096, 8, 128
    if torch.cuda.mem_get_info(dev)[0] < 5 * slots * heads * dim:
        pytest.skip("not enough memory")
    k = torch.empty((slots, heads, dim), dtype=BF, device=dev)
    v = torch.empty((slots, heads, dim), dtype=BF, device=dev)
    b = Batch([256, 200], 2, 8, heads, dim, 64, BF, seed=41)
    table = b.table.clone()
    for i in range(2):
        for c in range(table.shape[1]):
            old = int(b.table[i, c])
            table[i, c] = slots // 64 - 1 - (i * table.shape[1] + c)
            for t, s in ((k, b.kv[0]), (v, b.kv[1])):
                t[int(table[i, c]) * 64:][:64] = s[old * 64:old * 64 + 64].to(dev)
    out, lse = gb.tree_attention(b.q.to(dev), k, v, table.to(dev), b.lens.to(dev), page_size=64, next_n=2,
                                 return_lse=True)
    torch.cuda.synchronize(dev)
    rows, lens = b.table.numpy(), b.lens.numpy()
    check_rows(b, out, lse, lambda r: ref.visible(rows, 64, b.kv.shape[1], lens, 2, None, r))
    idx = torch.full((4, 96), -1, dtype=torch.int32)
    small = torch.full((4, 96), -1, dtype=torch.int32)
    for r in range(4):
        for j in range(0, 96, 2):
            p = (j * 7 + r) % 200
            idx[r, j] = int(table[r // 2, p // 64]) * 64 + p % 64
            small[r, j] = int(b.table[r // 2, p // 64]) * 64 + p % 64
    out, lse = gb.selected_attention(b.q.to(dev), k, v, idx.to(dev), return_lse=True)
    torch.cuda.synchronize(dev)
    check_rows(b, out, lse, lambda r: ref.selected(small.numpy(), b.kv.shape[1], r))


def test_tree_attention_long_context_split(dev):
    """One request, a long context: the work of one head is shared by many
    blocks and joined."""
    b = Batch([20011], 2, 4, 1, 64, 64, BF, seed=77)
    check_tree(dev, b)


def test_tree_attention_graph_replay_and_side_stream(dev):
    b = Batch([300, 270, 150], 2, 4, 2, 64, 16, BF, seed=5)
    k, v = b.caches(dev)
    q, table, lens = b.q.to(dev), b.table.to(dev), b.lens.to(dev)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        q2 = torch.empty_like(q)
        q2.copy_(q)                 # produced on this stream just before
        gb.tree_attention(q2, k, v, table, lens, page_size=16, next_n=2, return_lse=True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, lse = gb.tree_attention(q2, k, v, table, lens, page_size=16, next_n=2, return_lse=True)
    torch.cuda.synchronize(dev)
    for new in ([300, 270, 150], [17, 0, 149], [1, 256, 2]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize(dev)
        b.lens = torch.tensor(new, dtype=torch.int32)
        check_rows(b, out, lse, lambda r: ref.visible(b.table.numpy(), 16, k.shape[0], b.lens.numpy(), 2, None, r))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows,top_k,q_heads,kv_heads,dim", [
    (1, 1, 1, 1, 64), (5, 130, 8, 2, 128), (9, 257, 16, 1, 96), (3, 64, 7, 7, 8), (4, 300, 6, 2, 256), (2, 1500, 32, 4, 64),
    (2, 200, 128, 1, 128), (2, 150, 160, 1, 72),
])
def test_selected_attention(dev, dtype, rows, top_k, q_heads, kv_heads, dim):
    b = Batch([600], 1, q_heads, kv_heads, dim, 1, dtype, seed=rows + dim)
    g = torch.Generator().manual_seed(top_k)
    b.q = torch.randn((rows, q_heads, dim), generator=g).to(dtype)
    k, v = b.caches(dev)
    idx = b.table[0][torch.randint(0, 600, (rows, top_k), generator=g)]
    idx[torch.rand(idx.shape, generator=g) < 0.2] = -1          # holes anywhere
    if rows > 2:
        idx[1] = -1                                             # nothing selected
        idx[2, -1] = k.shape[0]                                 # beyond the cache
        idx[2, 0] = 2 ** 31 - 1
    buf = torch.full((rows, top_k + 3), 0, dtype=torch.int32)
    buf[:, :top_k] = idx
    out, lse = gb.selected_attention(b.q.to(dev), k, v, buf.to(dev)[:, :top_k], return_lse=True)
    torch.cuda.synchronize(dev)
    check_rows(b, out, lse, lambda r: ref.selected(idx.numpy(), k.shape[0], r))


def test_selected_attention_reads_the_transforms_output(dev):
    """The slots of top_k_page_table_transform, straight into the attention."""
    b = Batch([900, 1024, 3], 1, 8, 2, 128, 64, BF, seed=19)
    g = torch.Generator().manual_seed(8)
    scores = torch.randn((3, 1024), generator=g).to(dev)
    k, v = b.caches(dev)
    idx = gb.top_k_page_table_transform(scores, b.lens.to(dev), b.table.to(dev), 256, page_size=64)
    out, lse = gb.selected_attention(b.q.to(dev), k, v, idx, return_lse=True)
    torch.cuda.synchronize(dev)
    check_rows(b, out, lse, lambda r: ref.selected(idx.cpu().numpy(), k.shape[0], r))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,next_n,q_heads,kv_heads,dim,page,tree,shared,accept", [
    ([1], 1, 1, 1, 64, 1, False, True, False),
    ([200, 0, 129, 3], 4, 8, 2, 128, 16, True, False, True),
    ([140, 64], 64, 4, 2, 64, 7, True, True, True),
    ([260, 30], 33, 16, 2, 96, 64, True, False, False),
    ([150, 8], 2, 12, 4, 256, 32, False, True, False),
    ([90], 3, 5, 5, 8, 100, True, False, True),
])
def test_accumulate_cache_weights(dev, dtype, lens, next_n, q_heads, kv_heads, dim, page, tree, shared, accept):
    b = Batch(lens, next_n, q_heads, kv_heads, dim, page, dtype, seed=dim + next_n, fused=dim == 64)
    k, v = b.caches(dev)
    mask = trees(len(lens), next_n, 6) if tree else None
    dmask = None if mask is None else torch.from_numpy(mask).to(dev)
    _, lse = gb.tree_attention(b.q.to(dev), k, v, b.table.to(dev), b.lens.to(dev), page_size=page, next_n=next_n,
                               tree_mask=dmask, return_lse=True)
    took = np.random.RandomState(3).randint(-2 ** 63, 2 ** 63 - 1, len(lens)) if accept else None
    g = torch.Generator().manual_seed(1)
    width = b.table.shape[1] * page + 5 if dim != 96 else 201        # one narrower than the lengths
    w = torch.rand((len(lens), 1 if shared else kv_heads, width), generator=g)
    wd = w.to(dev)
    got = gb.accumulate_cache_weights(b.q.to(dev), k, lse, b.table.to(dev), b.lens.to(dev), wd, page_size=page,
                                      next_n=next_n, tree_mask=dmask,
                                      accept_mask=None if took is None else torch.from_numpy(took).to(dev))
    torch.cuda.synchronize(dev)
    assert got.data_ptr() == wd.data_ptr()
    q, kk, _ = b.wide()
    want, tol = ref.weights(q, kk, lse.cpu().numpy(), w.numpy(), b.table.numpy(), page, k.shape[0], b.lens.numpy(), next_n,
                            mask, took, b.group, b.scale)
    off = np.abs(got.cpu().double().numpy() - want)
    assert np.all(off <= tol), np.max(off - tol)


def test_accumulated_weights_of_a_row_sum_to_its_heads(dev):
    """Each row hands out one unit a head; the same call twice adds twice,
    to the bit the same amounts."""
    b = Batch([513], 1, 8, 2, 64, 16, BF, seed=4)
    k, v = b.caches(dev)
    args = (b.q.to(dev), k)
    _, lse = gb.tree_attention(*args, v, b.table.to(dev), b.lens.to(dev), page_size=16, return_lse=True)
    runs = [gb.accumulate_cache_weights(*args, lse, b.table.to(dev), b.lens.to(dev), torch.zeros((1, 1, 600), device=dev),
                                        page_size=16) for _ in range(2)]
    assert abs(float(runs[0].double().sum()) - 8) < 8 * 1e-4
    assert torch.equal(runs[0], runs[1]) and not runs[0][0, 0, 513:].any()


def moved(b, kept, dev, k, v):
    """Where every kept row has to be, on the CPU."""
    want = b.kv.clone()
    k0, v0 = (b.kv[:, 0], b.kv[:, 1]) if b.fused else (b.kv[0], b.kv[1])
    k1, v1 = (want[:, 0], want[:, 1]) if b.fused else (want[0], want[1])
    for i, rows in enumerate(kept):
        for h in range(k0.shape[1]):
            for j, p in enumerate(rows[h if len(rows) > 1 else 0]):
                dst = ref.slot_of(b.new_table[i].numpy(), b.page, k0.shape[0], j)
                src = ref.slot_of(b.table[i].numpy(), b.page, k0.shape[0], p)
                if dst >= 0:
                    k1[dst, h] = k0[src, h] if src >= 0 else 0
                    v1[dst, h] = v0[src, h] if src >= 0 else 0
    return k1, v1


def same_bits(a, b):
    it = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(it), b.contiguous().view(it))


@pytest.mark.parametrize("lens,next_n,kv_heads,dim,page,budget,recent,shared,accept,dtype", [
    ([1], 1, 1, 64, 1, 1, 0, True, False, BF),
    ([500, 0, 64, 63, 65], 1, 2, 64, 16, 64, 8, False, False, BF),
    ([500, 3, 64, 70, 71], 8, 4, 128, 7, 64, 64, False, True, HF),        # the recent ones alone
    ([900, 130, 128], 16, 2, 96, 64, 128, 200, True, True, BF),           # recent above the budget
    ([5000, 4097], 64, 1, 8, 100, 2048, 0, True, True, torch.float32),
    ([9001], 4, 2, 16, 32, 8192, 1000, False, True, HF),
    ([40], 4, 2, 16, 32, 64, 10, False, True, HF),                        # under its budget: drafts alone go
])
@pytest.mark.parametrize("kind", ["random", "ties", "special"])
def test_evict_cache(dev, lens, next_n, kv_heads, dim, page, budget, recent, shared, accept, dtype, kind):
    b = Batch(lens, next_n, kv_heads, kv_heads, dim, page, torch.float16 if dtype == torch.float32 else dtype,
              seed=budget, fused=dim == 64, spare=budget)
    if dtype == torch.float32:
        b.kv = torch.randn(b.kv.shape, generator=torch.Generator().manual_seed(2))
    g = torch.Generator().manual_seed(len(lens))
    width = max(lens) + 3
    w = torch.empty((len(lens), 1 if shared else kv_heads, width)).exponential_(generator=g)
    if kind == "ties":
        w = (w * 2).floor() / 2
    if kind == "special":
        pick = torch.rand(w.shape, generator=g)
        w[pick < 0.3] = 0.0
        w[pick < 0.15] = -0.0
        w[pick > 0.9] = math.inf
        w[pick > 0.95] = 1e-42
        w[(pick > 0.5) & (pick < 0.55)] = -1.0
    took = np.random.RandomState(8).randint(-2 ** 63, 2 ** 63 - 1, len(lens)) if accept else None
    k, v = b.caches(dev)
    got = gb.evict_cache(w.to(dev), k, v, b.table.to(dev), b.lens.to(dev), b.new_table.to(dev), budget, recent=recent,
                         page_size=page, next_n=next_n, accept_mask=None if took is None else torch.from_numpy(took).to(dev))
    torch.cuda.synchronize(dev)
    want = ref.evict(w.numpy(), b.lens.numpy(), b.table.numpy(), page, next_n, took, budget, recent)
    kept, weights = got.kept.cpu(), got.weights.cpu()
    for i, rows in enumerate(want):
        assert int(got.new_lens[i]) == len(rows[0])
        for h, keep in enumerate(rows):
            m = len(keep)
            assert kept[i, h, :m].tolist() == keep and (kept[i, h, m:] == -1).all()
            assert torch.equal(weights[i, h, :m], w[i, h, torch.tensor(keep, dtype=torch.long)])
            assert not weights[i, h, m:].any()
    k1, v1 = moved(b, want, dev, k, v)
    assert same_bits(k.cpu(), k1) and same_bits(v.cpu(), v1)


def test_evict_cache_missing_pages(dev):
    """A kept row without a source is zero; one without a destination is not written."""
    b = Batch([64, 64], 1, 2, 2, 64, 8, BF, seed=6, spare=32)
    b.table[0, 1] = -1
    b.new_table[1, 0] = -1
    w = torch.zeros((2, 1, 64))
    w[:, :, 8:24] = 1.0
    k, v = b.caches(dev)
    gb.evict_cache(w.to(dev), k, v, b.table.to(dev), b.lens.to(dev), b.new_table.to(dev), 32, recent=4, page_size=8)
    torch.cuda.synchronize(dev)
    k1, v1 = moved(b, ref.evict(w.numpy(), b.lens.numpy(), b.table.numpy(), 8, 1, None, 32, 4), dev, k, v)
    assert same_bits(k.cpu(), k1) and same_bits(v.cpu(), v1)


def test_evict_cache_long_rows(dev):
    """Weights of a row beyond what one block can hold, many of them equal."""
    n, budget = 400001, 1111
    g = torch.Generator().manual_seed(12)
    w = (torch.empty((2, 1, n)).exponential_(generator=g) * 64).floor()
    cols = -(-n // 64)
    table = torch.zeros((2, cols), dtype=torch.int32)
    new = torch.arange(2 * 18, dtype=torch.int32).view(2, 18) + 1
    k = torch.zeros((64 * 40, 1, 8), dtype=BF)
    lens = torch.tensor([n, n // 3], dtype=torch.int32)
    got = gb.evict_cache(w.to(dev), k.to(dev), k.to(dev), table.to(dev), lens.to(dev), new.to(dev), budget, recent=100,
                         page_size=64)
    for i, rows in enumerate(ref.evict(w.numpy(), lens.numpy(), table.numpy(), 64, 1, None, budget, 100)):
        assert got.kept[i, 0].tolist() == rows[0]
    assert got.new_lens.tolist() == [budget, budget]


def verify_inputs(requests, next_n, vocab, dtype, seed, tree):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((requests * next_n, vocab), generator=g) * 1.5
    hot = torch.randint(0, vocab, (requests * next_n, 3), generator=g)
    logits.scatter_add_(1, hot, torch.full(hot.shape, 6.0))
    mask = trees(requests, next_n, seed) if tree else None
    tokens = torch.zeros(requests * next_n, dtype=torch.int32)
    for i in range(requests):
        for n in range(1, next_n):
            above = n - 1 if mask is None else max(a for a in range(n) if ref.bits_of(mask[i * next_n + n]) >> a & 1)
            tokens[i * next_n + n] = hot[i * next_n + above, int(torch.randint(0, 3, (1,), generator=g))]
    noise = torch.empty((requests, vocab)).exponential_(generator=g).clamp_(min=1e-12)
    return logits.to(dtype), tokens, torch.rand(requests * next_n, generator=g), noise, mask


def check_verify(dev, logits, tokens, uniforms, noise, next_n, mask=None, temperature=None, draft=None):
    to = lambda t: None if t is None else t.to(dev)
    got = gb.verify_drafts(logits.to(dev), tokens.to(dev), uniforms.to(dev), noise.to(dev), next_n=next_n,
                           tree_mask=None if mask is None else torch.from_numpy(mask).to(dev), temperature=to(temperature),
                           draft_probs=to(draft))
    torch.cuda.synchronize(dev)
    want = ref.verify(logits.float().numpy(), tokens.numpy(), uniforms.numpy(), noise.numpy(), next_n, mask,
                      None if temperature is None else temperature.numpy(), None if draft is None else draft.numpy())
    for i, (count, path, follow, bits) in enumerate(want):
        assert int(got.accepted[i]) == count
        assert got.path[i].tolist() == path
        assert int(got.next_token[i]) == follow
        assert ref.bits_of(got.accept_mask[i]) == bits
    return want


@pytest.mark.parametrize("dtype", [torch.float32, BF, HF])
@pytest.mark.parametrize("requests,next_n,vocab,tree,temps", [
    (3, 1, 17, False, None),            # nothing drafted: a draw alone
    (1, 4, 1, False, None),             # one word
    (5, 4, 1000, False, "mixed"),
    (7, 16, 4099, True, "mixed"),
    (3, 64, 515, True, None),
    (2, 8, 40003, True, "greedy"),
])
def test_verify_drafts(dev, dtype, requests, next_n, vocab, tree, temps):
    logits, tokens, u, noise, mask = verify_inputs(requests, next_n, vocab, dtype, seed=vocab + next_n, tree=tree)
    temperature = {None: None, "greedy": torch.zeros(requests),
                   "mixed": torch.tensor([0.0, 0.7, 1.3, -1.0, 1.0, 0.5, 0.9])[:requests]}[temps]
    check_verify(dev, logits, tokens, u, noise, next_n, mask, temperature)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("vocab", [33, 5001])
def test_verify_drafts_against_draft_probabilities(dev, dtype, vocab):
    logits, tokens, u, noise, _ = verify_inputs(9, 5, vocab, dtype, seed=vocab, tree=False)
    g = torch.Generator().manual_seed(1)
    draft = torch.softmax(logits.float() + 0.7 * torch.randn(logits.shape, generator=g), 1)
    for i in range(9):
        for n in range(1, 5):
            tokens[i * 5 + n] = int(torch.multinomial(draft[i * 5 + n - 1], 1, generator=g))
    want = check_verify(dev, logits, tokens, u, noise, 5, None, torch.linspace(0.5, 1.5, 9), draft)
    assert len({w[0] for w in want}) > 1


def test_verify_drafts_odd_inputs(dev):
    """Repeated siblings, tokens outside the vocabulary, masked words, nodes
    without a parent, a row of nothing but -inf, uniforms of 0."""
    logits, tokens, u, noise, _ = verify_inputs(4, 6, 301, torch.float32, seed=3, tree=False)
    star = np.array([1] + [1 | 1 << n for n in range(1, 6)], dtype=np.int64)      # all children of the root
    mask = np.tile(star, 4)
    mask[6 + 2] = 1 << 2                                                          # no parent
    tokens[7:12] = tokens[7]
    u[6:12] = 0.999
    tokens[12 + 1], tokens[12 + 2] = -1, 301
    logits[12:18, 5:200] = -math.inf
    logits[18] = -math.inf
    u[0:6] = 0.0
    want = check_verify(dev, logits, tokens, u, noise, 6, mask)
    assert want[3][2] == -1 and want[0][0] == 1


def test_verify_drafts_strided_logits_and_ties(dev):
    """A padded row stride, a misaligned base, greedy rows whose largest
    logits are equal: the lowest index counts."""
    g = torch.Generator().manual_seed(9)
    x = torch.randint(-3, 4, (6, 1003), generator=g).to(BF)
    buf = torch.full((6, 1011), math.inf, dtype=BF, device=dev)
    buf[:, 3:1006] = x.to(dev)
    tokens = torch.zeros(6, dtype=torch.int32)
    noise = torch.ones((2, 1003))
    got = gb.verify_drafts(buf[:, 3:1006], tokens.to(dev), torch.zeros(6, device=dev), noise.to(dev), next_n=3,
                           temperature=torch.zeros(2, device=dev))
    want = ref.verify(x.float().numpy(), tokens.numpy(), np.zeros(6), noise.numpy(), 3, None, np.zeros(2))
    assert got.next_token.tolist() == [w[2] for w in want] and got.accepted.tolist() == [w[0] for w in want]


def test_verified_drafts_follow_the_target(dev):
    """The emitted token's law is the target's, whatever was drafted: 40000
    draws over 6 words.  A share has a deviation of at most sqrt(1/4/40000) =
    0.0025; 0.0125 is five of them."""
    n, vocab = 40000, 6
    g = torch.Generator().manual_seed(21)
    target = torch.tensor([0.05, 0.3, 0.1, 0.25, 0.2, 0.1])
    draft = torch.tensor([0.4, 0.1, 0.1, 0.1, 0.2, 0.1])
    logits = target.log().expand(2 * n, vocab).contiguous()
    for probs in (None, draft.expand(2 * n, vocab).contiguous()):
        drawn = torch.multinomial(draft, n, replacement=True, generator=g) if probs is not None else torch.ones(n, dtype=torch.long)
        tokens = torch.stack([torch.zeros(n, dtype=torch.long), drawn], 1).reshape(-1).to(torch.int32)
        noise = torch.empty((n, vocab)).exponential_(generator=g).clamp_(min=1e-12)
        got = gb.verify_drafts(logits.to(dev), tokens.to(dev), torch.rand(2 * n, generator=g).to(dev), noise.to(dev), next_n=2,
                               draft_probs=None if probs is None else probs.to(dev))
        first = torch.where(got.accepted.cpu() > 0, drawn, got.next_token.cpu().long())
        share = torch.bincount(first, minlength=vocab) / n
        assert float((share - target).abs().max()) < 0.0125


def test_empty_batches(dev):
    q = torch.empty((0, 4, 64), dtype=BF, device=dev)
    cache = torch.empty((8, 2, 64), dtype=BF, device=dev)
    table, lens = torch.empty((0, 3), dtype=torch.int32, device=dev), torch.empty(0, dtype=torch.int32, device=dev)
    assert gb.tree_attention(q, cache, cache, table, lens).shape == q.shape
    assert gb.selected_attention(q, cache, cache, table).shape == q.shape
    w = torch.empty((0, 2, 9), device=dev)
    assert gb.accumulate_cache_weights(q, cache, torch.empty((0, 4), device=dev), table, lens, w) is w
    assert gb.evict_cache(w, cache, cache, table, lens, table, 3).new_lens.numel() == 0
    x = torch.empty((0, 9), device=dev)
    assert gb.verify_drafts(x, lens, torch.empty(0, device=dev), x).accepted.numel() == 0
    # no columns at all: rows see nothing
    q = torch.ones((2, 4, 64), dtype=BF, device=dev)
    none = torch.empty((2, 0), dtype=torch.int32, device=dev)
    out, lse = gb.tree_attention(q, cache, cache, none, torch.tensor([5, 1], dtype=torch.int32, device=dev), return_lse=True)
    assert not out.any() and torch.isinf(lse).all()
    out, lse = gb.selected_attention(q, cache, cache, none, return_lse=True)
    assert not out.any() and torch.isinf(lse).all()
