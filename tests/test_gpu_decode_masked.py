"""Infinities and NaN in drafted tokens: they reach the rows that see the
token, as the formulas say, and no other row.

Tolerances where the definition is finite: as in test_gpu_decode."""
import math

import numpy as np
import pytest
import torch

import decode_reference as ref
import sparse_attention_top_gb300 as gb
from test_gpu_decode import BF, HF, Batch, trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def compare(b, out, lse, seen_of):
    """Finite entries within the bounds, the others of the same kind."""
    q, k, v = b.wide()
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    finite = 0
    for r in range(q.shape[0]):
        seen = seen_of(r)
        with np.errstate(invalid="ignore"):
            o, l, eta, mag = ref.attend(q[r], k, v, seen, b.group, b.scale)
        assert np.array_equal(np.isnan(l), np.isnan(lse[r])), r
        at = np.isfinite(o)
        finite += at.sum()
        with np.errstate(invalid="ignore"):
            tol = b.u * np.abs(o) + (b.u + 2 * eta[:, None]) * mag
            assert np.all(np.abs(out[r] - o)[at] <= tol[at]), r
        assert np.array_equal(np.isnan(o), np.isnan(out[r])), r
        assert np.array_equal(o[np.isinf(o)], out[r][np.isinf(o)]), r
        assert np.isfinite(out[r][at]).all()
        ok = np.isfinite(l)
        assert np.all(np.abs(lse[r][ok] - l[ok]) <= eta[ok] + 2.0 ** -21 * (1 + np.abs(l[ok])))
        assert np.array_equal(l == -math.inf, lse[r] == -math.inf)
    return finite


def draft_slot(b, i, j):
    p = int(b.lens[i]) - b.next_n + j
    return int(b.table[i, p // b.page]) * b.page + p % b.page


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,next_n,q_heads,kv_heads,dim,page,tree", [
    ([300, 5, 131, 129], 5, 8, 2, 128, 16, True),          # up to 32 rows a head
    ([40, 4], 4, 4, 1, 64, 8, False),                      # a chain, one without context
    ([260, 64, 100], 64, 2, 1, 128, 64, True),             # 128 rows a head; drafts across two tiles
    ([200, 170], 33, 16, 2, 96, 100, True),                # several row tiles
    ([150, 33], 7, 6, 2, 256, 32, True),                   # the largest dimension
    ([9000], 6, 4, 2, 72, 64, True),                       # shared by many blocks
    ([9000], 64, 4, 1, 64, 64, False),
    ([30] * 300, 4, 4, 2, 64, 16, True),                   # several units a block
])
@pytest.mark.parametrize("what", ["value", "key"])
def test_tree_attention_of_drafts_that_are_not_finite(dev, dtype, lens, next_n, q_heads, kv_heads, dim, page, tree, what):
    b = Batch(lens, next_n, q_heads, kv_heads, dim, page, dtype, seed=next_n + dim)
    mask = trees(len(lens), next_n, 13) if tree else None
    kind = 0 if what == "key" else 1
    for i in range(len(lens)):
        for n, j in enumerate({next_n - 1, next_n // 2, max(1, next_n // 3)}):
            s = draft_slot(b, i, j)
            if kind == 0:
                b.kv[0, s] = math.nan
            elif (i + n) % 3 == 0:
                b.kv[1, s, n % kv_heads, (5 * n + i) % dim] = -math.inf
            elif (i + n) % 3 == 1:
                b.kv[1, s, :, -1] = math.inf
            else:
                b.kv[1, s] = math.nan
    k, v = b.caches(dev)
    out, lse = gb.tree_attention(b.q.to(dev), k, v, b.table.to(dev), b.lens.to(dev), page_size=page, next_n=next_n,
                                 tree_mask=None if mask is None else torch.from_numpy(mask).to(dev), return_lse=True)
    torch.cuda.synchronize(dev)
    table, at = b.table.numpy(), b.lens.numpy()
    assert compare(b, out, lse, lambda r: ref.visible(table, page, k.shape[0], at, next_n, mask, r)) > 0


@pytest.mark.parametrize("top_k", [40, 300, 5000])
def test_selected_attention_of_a_key_that_is_not_finite(dev, top_k):
    b = Batch([6000], 1, 8, 2, 64, 1, BF, seed=6)
    g = torch.Generator().manual_seed(top_k)
    b.q = torch.randn((3, 8, 64), generator=g).to(BF)
    idx = b.table[0][torch.stack([torch.randperm(5999, generator=g)[:top_k] for _ in range(3)])].clone()
    bad = int(b.table[0, 5999])
    b.kv[0, bad] = math.nan
    b.kv[1, bad] = math.nan
    idx[1, top_k // 2] = bad                   # one row selects it, its neighbours do not
    k, v = b.caches(dev)
    out, lse = gb.selected_attention(b.q.to(dev), k, v, idx.to(dev), return_lse=True)
    torch.cuda.synchronize(dev)
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert compare(b, out, lse, lambda r: ref.selected(idx.numpy(), k.shape[0], r)) == 2 * 8 * 64


def test_weights_of_keys_that_are_not_finite(dev):
    """A rejected draft's NaN adds nothing; a visible key's -infinity score adds
    nothing to its position, whatever rows the tile is filled up with."""
    b = Batch([140, 37], 4, 6, 2, 64, 16, BF, seed=15)
    mask = trees(2, 4, 4)
    mask[:] = torch.tensor([1, 3, 5, 11] * 2).numpy()              # node 2 is node 1's sibling
    took = np.array([0b1011, 0b1011])
    b.q[..., 0] = -1
    for i in range(2):
        b.kv[0, draft_slot(b, i, 2)] = math.nan
        s = int(b.table[i, 0]) * 16 + 3
        b.kv[0, s, :, 0] = math.inf
    k, v = b.caches(dev)
    args = dict(page_size=16, next_n=4, tree_mask=torch.from_numpy(mask).to(dev))
    _, lse = gb.tree_attention(b.q.to(dev), k, v, b.table.to(dev), b.lens.to(dev), return_lse=True, **args)
    w = torch.rand((2, 2, 144), generator=torch.Generator().manual_seed(2))
    got = gb.accumulate_cache_weights(b.q.to(dev), k, lse, b.table.to(dev), b.lens.to(dev), w.to(dev),
                                      accept_mask=torch.from_numpy(took).to(dev), **args)
    torch.cuda.synchronize(dev)
    got = got.cpu()
    assert torch.isfinite(got).all()
    for i in range(2):
        p = int(b.lens[i]) - 2
        assert torch.equal(got[i, :, p], w[i, :, p])
        assert torch.equal(got[i, :, 3], w[i, :, 3])
    b.kv[0, int(b.table[0, 0]) * 16 + 3] = 0     # the definition over the other positions
    b.kv[0, int(b.table[1, 0]) * 16 + 3] = 0
    q, kk, _ = b.wide()
    want, tol = ref.weights(q, np.nan_to_num(kk), lse.cpu().numpy(), w.numpy(), b.table.numpy(), 16, k.shape[0],
                            b.lens.numpy(), 4, mask, took, b.group, b.scale)
    rest = np.ones(144, dtype=bool)
    rest[3] = False
    off = np.abs(got.double().numpy() - want)
    assert np.all((off <= tol)[:, :, rest]), np.max((off - tol)[:, :, rest])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("next_n,q_heads,kv_heads,dim,shared", [(2, 4, 2, 64, False), (20, 4, 2, 128, True), (64, 6, 2, 256, False)])
def test_weights_of_rows_without_a_sum(dev, dtype, next_n, q_heads, kv_heads, dim, shared):
    """A row whose lse is -infinity adds nothing, whatever the keys hold."""
    b = Batch([300, 170], next_n, q_heads, kv_heads, dim, 16, dtype, seed=next_n)
    for i in range(2):
        for p, x in ((10, math.nan), (20, math.inf), (131, -math.inf)):
            b.kv[0, int(b.table[i, p // 16]) * 16 + p % 16] = x
    k, _ = b.caches(dev)
    w = torch.rand((2, 1 if shared else kv_heads, 300), generator=torch.Generator().manual_seed(2))
    lse = torch.full((2 * next_n, q_heads), -math.inf)
    for accept in (None, torch.tensor([1, 3])):
        got = gb.accumulate_cache_weights(b.q.to(dev), k, lse.to(dev), b.table.to(dev), b.lens.to(dev), w.to(dev), page_size=16,
                                          next_n=next_n, accept_mask=None if accept is None else accept.to(dev))
        assert torch.equal(got.cpu(), w)
    # beside rows that have one: request 1 alone keeps its lse, over finite keys
    for p in (10, 20, 131):
        b.kv[0, int(b.table[1, p // 16]) * 16 + p % 16] = 0.5
    k, v = b.caches(dev)
    full = gb.tree_attention(b.q.to(dev), k, v, b.table.to(dev), b.lens.to(dev), page_size=16, next_n=next_n, return_lse=True)[1]
    lse[next_n:] = full[next_n:].cpu()
    lse[next_n, 0] = -math.inf
    got = gb.accumulate_cache_weights(b.q.to(dev), k, lse.to(dev), b.table.to(dev), b.lens.to(dev), w.to(dev), page_size=16,
                                      next_n=next_n).cpu()
    assert torch.equal(got[0], w[0])
    q, kk, _ = b.wide()
    want, tol = ref.weights(q[next_n:], kk, lse.numpy()[next_n:], w.numpy()[1:], b.table.numpy()[1:], 16, k.shape[0],
                            b.lens.numpy()[1:], next_n, None, None, b.group, b.scale)
    off = np.abs(got[1:].double().numpy() - want)
    assert np.all(off <= tol), np.max(off - tol)
