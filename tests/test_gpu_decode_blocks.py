"""Decode-step operators where a block has several tiles, several units or a
part of one, against plain float64 products on the GPU; and their bounded waits.

Tolerances as in test_gpu_decode: u |out| + (u + 2 eta) sum p |v| with u the
16-bit type's unit roundoff and eta the bound on a score's error.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
sys.path[:0] = [p for p in (ROOT, HERE) if p not in sys.path]   # as a child process too

import decode_reference as ref  # noqa: E402
import sparse_attention_top_gb300 as gb  # noqa: E402

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def make(dev, lens, next_n, q_heads, kv_heads, dim, page, dtype, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    b, cols = len(lens), max(1, -(-max(lens) // page))
    order = torch.randperm(b * cols, generator=g, device=dev).to(torch.int32)
    k = torch.randn((b * cols * page, kv_heads, dim), generator=g, device=dev).to(dtype)
    v = torch.randn(k.shape, generator=g, device=dev).to(dtype)
    q = torch.randn((b * next_n, q_heads, dim), generator=g, device=dev).to(dtype)
    return q, k, v, order.view(b, cols), torch.tensor(lens, dtype=torch.int32, device=dev)


def attend(q, k, v, scale):
    """[rows, heads of a group, dim] over [n, dim]: out, lse, eta, sum p |v|."""
    s = torch.einsum("tgd,nd->tgn", q.double(), k.double()) * scale
    lse = torch.logsumexp(s, 2)
    p = torch.exp(s - lse.unsqueeze(2))
    size = torch.einsum("tgd,nd->tgn", q.double().abs(), k.double().abs()).amax(2) * abs(scale)
    eta = (q.shape[2] + 8) * 2.0 ** -23 * size + 2.0 ** -20
    return torch.einsum("tgn,nd->tgd", p, v.double()), lse, eta, torch.einsum("tgn,nd->tgd", p, v.double().abs())


def check(out, lse, want, u):
    o, l, eta, mag = want
    tol = u * o.abs() + (u + 2 * eta.unsqueeze(2)) * mag
    assert bool(((out.double() - o).abs() <= tol).all()), float(((out.double() - o).abs() - tol).max())
    assert bool(((lse.double() - l).abs() <= eta + 2.0 ** -21 * (1 + l.abs())).all())


def check_tree(dev, lens, next_n, q_heads, kv_heads, dim, page, dtype, seed=1, scale=None):
    q, k, v, table, n = make(dev, lens, next_n, q_heads, kv_heads, dim, page, dtype, seed)
    out, lse = gb.tree_attention(q, k, v, table, n, page_size=page, next_n=next_n, scale=scale, return_lse=True)
    torch.cuda.synchronize(dev)
    g, u, scale = q_heads // kv_heads, ref.U[str(dtype).replace("torch.", "")], dim ** -0.5 if scale is None else scale
    for i, length in enumerate(lens):
        if length == 0:
            assert not out[i * next_n:(i + 1) * next_n].any() and bool(torch.isneginf(lse[i * next_n:(i + 1) * next_n]).all())
        pos = torch.arange(length, device=dev)
        slots = table[i, pos // page].long() * page + pos % page
        for t in range(next_n):
            seen = slots[:max(0, length - next_n + t + 1)]
            if not seen.numel():
                continue
            r = i * next_n + t
            for h in range(kv_heads):
                heads = slice(h * g, h * g + g)
                check(out[r:r + 1, heads], lse[r:r + 1, heads], attend(q[r:r + 1, heads], k[seen, h], v[seen, h], scale), u)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,next_n,q_heads,kv_heads,dim,page", [
    ([256], 1, 152, 152, 64, 64),                     # two tiles of every unit, a unit a block
    ([384], 1, 160, 160, 128, 16),                    # three, and more units than blocks
    ([130, 0, 700, 1, 0, 390], 2, 96, 48, 128, 7),    # short, long and empty units in one block
    ([513, 260], 3, 160, 20, 64, 128),                # 24 rows a unit
    ([700, 300], 8, 96, 12, 128, 32),                 # 64 rows: the warpgroups share them
    ([640, 257], 16, 64, 4, 128, 1),                  # 256 rows: a row tile each
    ([500, 129], 5, 224, 4, 64, 64),                  # 280 rows: two row tiles, the second short
    ([700, 260, 65], 2, 48, 24, 256, 16),             # dimension 256
    ([8000], 20, 16, 2, 256, 64),                     # 160 rows of it, split over blocks
    ([9000, 40], 4, 8, 1, 200, 100),
])
def test_tree_attention_units_and_tiles_of_a_block(dev, dtype, lens, next_n, q_heads, kv_heads, dim, page):
    check_tree(dev, lens, next_n, q_heads, kv_heads, dim, page, dtype)


@pytest.mark.parametrize("scale", [-0.11, 0.0, 1.7])
def test_tree_attention_scales(dev, scale):
    """A negative scale, none at all (the mean of the values), a steep one."""
    check_tree(dev, [1000, 140], 2, 8, 2, 64, 16, BF, seed=3, scale=scale)


def test_tree_attention_rising_maximum(dev):
    """Each tile's scores far above the one's before: O is rescaled."""
    q, k, v, table, n = make(dev, [2000], 1, 8, 2, 128, 64, HF, 9)
    steps = (torch.arange(2000, device=dev) // 100).to(HF)
    slots = table[0, torch.arange(2000, device=dev) // 64].long() * 64 + torch.arange(2000, device=dev) % 64
    k[slots] = (q[0, ::4].sign() * 0.5).unsqueeze(0) * steps.view(-1, 1, 1) + 0.1 * k[slots]
    out, lse = gb.tree_attention(q, k, v, table, n, page_size=64, return_lse=True)
    for h in range(2):
        heads = slice(h * 4, h * 4 + 4)
        check(out[:, heads], lse[:, heads], attend(q[:, heads], k[slots, h], v[slots, h], 128 ** -0.5), ref.U["float16"])


@pytest.mark.parametrize("rows,top_k,q_heads,kv_heads,dim", [(200, 316, 32, 2, 128), (40, 2048, 16, 1, 64), (90, 700, 48, 1, 96),
                                                            (3, 5000, 256, 1, 128)])
def test_selected_attention_units_and_tiles_of_a_block(dev, rows, top_k, q_heads, kv_heads, dim):
    g = torch.Generator(device=dev).manual_seed(top_k)
    k = torch.randn((9000, kv_heads, dim), generator=g, device=dev).to(BF)
    v = torch.randn(k.shape, generator=g, device=dev).to(BF)
    q = torch.randn((rows, q_heads, dim), generator=g, device=dev).to(BF)
    idx = torch.randint(0, 9000, (rows, top_k), generator=g, device=dev, dtype=torch.int32)
    count = torch.randint(0, top_k + 1, (rows, 1), generator=g, device=dev)
    count[::3] = top_k
    idx = torch.where(torch.arange(top_k, device=dev) < count, idx, -1)
    out, lse = gb.selected_attention(q, k, v, idx, return_lse=True)
    group = q_heads // kv_heads
    for r in range(rows):
        at = idx[r][idx[r] >= 0].long()
        if not at.numel():
            assert not out[r].any() and bool(torch.isneginf(lse[r]).all())
            continue
        for h in range(kv_heads):
            heads = slice(h * group, h * group + group)
            check(out[r:r + 1, heads], lse[r:r + 1, heads], attend(q[r:r + 1, heads], k[at, h], v[at, h], dim ** -0.5),
                  ref.U["bfloat16"])


@pytest.mark.parametrize("lens,next_n,q_heads,kv_heads,dim,shared", [
    ([5000, 1, 0, 300], 2, 64, 16, 128, False), ([3000, 900], 4, 32, 8, 64, True), ([2600, 140], 40, 16, 2, 128, True),
    ([2500, 260], 3, 20, 10, 256, False), ([4100], 33, 16, 2, 256, True),
])
def test_accumulate_cache_weights_units_and_tiles_of_a_block(dev, lens, next_n, q_heads, kv_heads, dim, shared):
    page = 32
    q, k, v, table, n = make(dev, lens, next_n, q_heads, kv_heads, dim, page, BF, 5)
    _, lse = gb.tree_attention(q, k, v, table, n, page_size=page, next_n=next_n, return_lse=True)
    took = torch.tensor([(0x5A5A5A5A5 * (i + 3)) & ((1 << next_n) - 1) for i in range(len(lens))], device=dev)
    w = torch.rand((len(lens), 1 if shared else kv_heads, max(lens)), device=dev)
    want, tol = w.double(), w.double() * 2.0 ** -23
    got = gb.accumulate_cache_weights(q, k, lse, table, n, w.clone(), page_size=page, next_n=next_n, accept_mask=took)
    g, scale = q_heads // kv_heads, dim ** -0.5
    for i, length in enumerate(lens):
        pos = torch.arange(length, device=dev)
        slots = table[i, pos // page].long() * page + pos % page
        for t in range(next_n):
            if not int(took[i]) >> t & 1:
                continue
            m = max(0, length - next_n + t + 1)
            for h in range(kv_heads):
                rows = q[i * next_n + t, h * g:h * g + g].double()
                kk = k[slots[:m], h].double()
                at = lse[i * next_n + t, h * g:h * g + g].double().unsqueeze(1)
                eta = (dim + 8) * 2.0 ** -23 * scale * (rows.abs() @ kk.abs().T) + 2.0 ** -20
                p = torch.exp(scale * (rows @ kk.T) - at)
                want[i, 0 if shared else h, :m] += p.sum(0)
                tol[i, 0 if shared else h, :m] += (p * (1.5 * eta + at.abs() * 2.0 ** -22 + q_heads * next_n * 2.0 ** -23)).sum(0)
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


def test_cache_weights_and_eviction_beyond_32_bits(dev):
    """Slots whose element offset passes 2^32, read for the weights and moved."""
    slots, heads, dim = (1 << 32) // 1024 + 4096, 8, 128
    if torch.cuda.mem_get_info(dev)[0] < 5 * slots * heads * dim:
        pytest.skip("not enough memory")
    k = torch.empty((slots, heads, dim), dtype=BF, device=dev)
    v = torch.empty((slots, heads, dim), dtype=BF, device=dev)
    last = slots // 64 - 1
    table = torch.tensor([[last, 3, last - 1, last - 2]], dtype=torch.int32, device=dev)
    new = torch.tensor([[last - 3, last - 4]], dtype=torch.int32, device=dev)
    pos = torch.arange(256, device=dev)
    at = table[0, pos // 64].long() * 64 + pos % 64
    k[at] = torch.randn((256, heads, dim), device=dev).to(BF)
    v[at] = torch.randn((256, heads, dim), device=dev).to(BF)
    q = torch.randn((1, heads, dim), device=dev).to(BF)
    n = torch.tensor([256], dtype=torch.int32, device=dev)
    _, lse = gb.tree_attention(q, k, v, table, n, page_size=64, return_lse=True)
    w = gb.accumulate_cache_weights(q, k, lse, table, n, torch.zeros((1, heads, 256), device=dev), page_size=64)
    p = torch.softmax(torch.einsum("hd,nhd->hn", q[0].double(), k[at].double()) * dim ** -0.5, 1)
    assert bool(((w[0].double() - p).abs() <= 1e-3 * p).all())
    got = gb.evict_cache(w, k, v, table, n, new, 100, recent=20, page_size=64)
    to = new[0, torch.arange(100, device=dev) // 64].long() * 64 + torch.arange(100, device=dev) % 64
    kept = ref.evict(w.cpu().numpy(), [256], table.cpu().numpy(), 64, 1, None, 100, 20)[0]
    for h in range(heads):
        assert got.kept[0, h].tolist() == kept[h]
        assert torch.equal(k[to, h], k[at[kept[h]], h]) and torch.equal(v[to, h], v[at[kept[h]], h])


@pytest.mark.parametrize("dtype", [torch.float32, BF, HF])
def test_verify_drafts_of_a_large_batch(dev, dtype):
    """Batches whose rows are read as the walk reaches them."""
    import test_gpu_decode as small
    logits, tokens, u, noise, mask = small.verify_inputs(110, 4, 50021, dtype, seed=17, tree=True)
    temperature = torch.linspace(-0.2, 1.4, 110)
    want = small.check_verify(dev, logits, tokens, u, noise, 4, mask, temperature)
    assert len({w[0] for w in want}) > 2
    draft = torch.softmax(logits.float() + 0.5, 1)
    small.check_verify(dev, logits, tokens, u, noise, 4, None, temperature, draft)


def _child():
    """A process whose waits run out after the first try (which itself waits a
    while, so not every call's do): every call comes back, and one that gave
    up says in the status word that its outputs are not reliable."""
    d = torch.device("cuda:0")
    gave_up = {"attention": 0, "weights": 0}
    for next_n, q_heads in ((1, 4), (4, 32), (8, 64)):
        for dim in (64, 128, 256):
            q, k, v, table, n = make(d, [30000, 20000], next_n, q_heads, 4, dim, 16, BF, 2)
            ws = torch.zeros(gb.gbtopk_attention_workspace_bytes(q.shape[0], q_heads, 4, dim), dtype=torch.uint8, device=d)
            _, lse = gb.tree_attention(q, k, v, table, n, page_size=16, next_n=next_n, return_lse=True, workspace=ws)
            torch.cuda.synchronize(d)
            status = gb.gbtopk_device_status(ws)
            assert status in (0, 2) and gb.gbtopk_device_status(ws) == 0
            gave_up["attention"] += status == 2
            w = torch.zeros((2, 4, 30000), device=d)
            gb.accumulate_cache_weights(q, k, lse, table, n, w, page_size=16, next_n=next_n, workspace=ws)
            torch.cuda.synchronize(d)
            status = gb.gbtopk_device_status(ws)
            assert status in (0, 2)
            gave_up["weights"] += status == 2
    assert gave_up["attention"] and gave_up["weights"], gave_up
    print("child: ok", gave_up)


def test_waits_that_run_out_end_the_call(dev):
    env = dict(os.environ, GBTOPK_WAIT_POLLS="1")
    r = subprocess.run([sys.executable, os.path.abspath(__file__), "child"], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "child: ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
    print(r.stdout)


if __name__ == "__main__" and len(sys.argv) > 1 and sys.argv[1] == "child":
    _child()
