"""Attention where one key outweighs the others by many powers of e, as an
attention sink does, and its value is zero: the output is the others' part.

Tolerances: as in test_gpu_decode_blocks (u |out| + (u + 2 eta) sum p |v|), and
for fp16, whose smallest number is 2^-24: half of it for the output, and for
each probability of a tile half of it under the tile's own scale, which puts
the tile's largest probability at 2^-1 or above, and at 2^6.5 or above where
that is the row's largest."""
import pytest
import torch

import decode_reference as ref
import sparse_attention_top_gb300 as gb
from test_gpu_decode import BF, HF

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def check(out, lse, q, k, v, dtype):
    """[heads, dim] rows over [n, dim], one score scale: 1."""
    s = q.double() @ k.double().T
    want_lse = torch.logsumexp(s, 1)
    p = torch.exp(s - want_lse.unsqueeze(1))
    o, mag = p @ v.double(), p @ v.double().abs()
    u = ref.U[str(dtype).replace("torch.", "")]
    eta = (q.shape[1] + 8) * 2.0 ** -23 * (q.double().abs() @ k.double().abs().T).amax(1) + 2.0 ** -20
    tol = u * o.abs() + (u + 2 * eta.unsqueeze(1)) * mag
    if dtype == HF:
        tile = 64 if q.shape[1] > 128 else 128
        tops = torch.nn.functional.pad(p, (0, -p.shape[1] % tile)).view(p.shape[0], -1, tile).amax(2)
        first = tops == tops.amax(1, keepdim=True)
        unit = torch.where(first, tops * 2.0 ** -6.5, tops * 2.0).sum(1)
        tol = tol + 2.0 ** -25 + tile * 2.0 ** -25 * (unit * v.double().abs().max()).unsqueeze(1)
    off = (out.double() - o).abs()
    assert bool((off <= tol).all()), (float((off - tol).max()), float((off / o.abs().clamp(min=2.0 ** -24)).max()))
    off = (lse.double() - want_lse).abs()
    assert bool((off <= eta + 2.0 ** -21 * (1 + want_lse.abs())).all()), float(off.max())


def levels(kind, gap, n, g, dev):
    """Scores in nats, multiples of 1/8, below 64: one sink, or many of all heights."""
    at = torch.randint(-2, 3, (n,), generator=g, device=dev) / 8.0
    zero = torch.zeros(n, dtype=torch.bool, device=dev)
    if kind == "first":
        zero[0] = True
    elif kind == "middle":
        zero[n // 2] = True
    else:           # the reference rises and falls again and again
        zero[torch.randint(0, n, (n // 700 + 1,), generator=g, device=dev)] = True
    at[zero] = gap if kind != "many" else (torch.rand(int(zero.sum()), generator=g, device=dev) * gap * 8).round() / 8
    return at, zero


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("next_n,q_heads,kv_heads,dim,n", [
    (1, 8, 2, 128, 20011),      # up to 32 rows a head
    (3, 8, 1, 64, 9000),
    (9, 16, 2, 128, 9000),      # up to 128
    (40, 8, 1, 64, 5000),       # several row tiles
    (17, 32, 2, 128, 5000),
    (5, 12, 2, 256, 9000),      # one warpgroup
])
@pytest.mark.parametrize("kind,gap,value", [("first", 12, 1), ("first", 18, 1), ("middle", 18, 1), ("first", 24, 64),
                                            ("middle", 30, 512), ("many", 20, 4), ("first", 50, 512)])
def test_tree_attention_with_a_sink(dev, dtype, next_n, q_heads, kv_heads, dim, n, kind, gap, value):
    g = torch.Generator(device=dev).manual_seed(gap + dim)
    at, zero = levels(kind, gap, n - next_n, g, dev)
    k = torch.zeros((n, kv_heads, dim), device=dev)
    k[:n - next_n, :, 3] = at.unsqueeze(1) / 8
    v = value * (1 + 0.25 * torch.randn(k.shape, generator=g, device=dev))
    v[:n - next_n][zero] = 0
    q = torch.zeros((next_n, q_heads, dim), device=dev)
    q[:, :, 3] = 8
    q[:, 1::2, 3] = 7          # the rows of a warp move apart
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    page = 16
    table = torch.arange(-(-n // page), dtype=torch.int32, device=dev).unsqueeze(0)
    pad = table.shape[1] * page - n
    kc, vc = (torch.cat([x, torch.zeros((pad, *x.shape[1:]), dtype=dtype, device=dev)]) for x in (k, v))
    out, lse = gb.tree_attention(q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device=dev), page_size=page,
                                 next_n=next_n, scale=1.0, return_lse=True)
    torch.cuda.synchronize(dev)
    group = q_heads // kv_heads
    for t in range(next_n):
        seen = n - next_n + t + 1
        for h in range(kv_heads):
            heads = slice(h * group, h * group + group)
            check(out[t, heads], lse[t, heads], q[t, heads], k[:seen, h], v[:seen, h], dtype)


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("kind,gap", [("first", 18), ("middle", 24), ("many", 20)])
def test_selected_attention_with_a_sink(dev, dtype, kind, gap):
    g = torch.Generator(device=dev).manual_seed(gap)
    n, heads, dim = 3000, 16, 128
    at, zero = levels(kind, gap, n, g, dev)
    k = torch.zeros((n, 1, dim), device=dev)
    k[:, 0, 3] = at / 8
    v = 32 * (1 + 0.25 * torch.randn(k.shape, generator=g, device=dev))
    v[zero] = 0
    q = torch.zeros((2, heads, dim), device=dev)
    q[:, :, 3] = 8
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    idx = torch.arange(n, dtype=torch.int32, device=dev).expand(2, n).contiguous()
    out, lse = gb.selected_attention(q, k, v, idx, scale=1.0, return_lse=True)
    torch.cuda.synchronize(dev)
    for r in range(2):
        check(out[r], lse[r], q[r], k[:, 0], v[:, 0], dtype)


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("next_n,dim", [(1, 64), (1, 128), (40, 128), (40, 256), (1, 256)])
def test_a_row_that_sees_one_token_is_its_value(dev, dtype, next_n, dim):
    """To the bit: its probability is one, whatever its score."""
    g = torch.Generator(device=dev).manual_seed(dim)
    n, heads = 30, 8
    q = torch.randn((n * next_n, heads, dim), generator=g, device=dev).to(dtype)
    k, v = torch.randn((2, n * next_n, 2, dim), generator=g, device=dev).to(dtype)
    table = torch.arange(n, dtype=torch.int32, device=dev).unsqueeze(1)
    lens = torch.full((n,), next_n, dtype=torch.int32, device=dev)
    alone = (1 << torch.arange(next_n, device=dev)).repeat(n)          # each token sees itself
    out = gb.tree_attention(q, k, v, table, lens, page_size=next_n, next_n=next_n, tree_mask=alone)
    assert torch.equal(out, v.repeat_interleave(heads // 2, 1))
    idx = torch.arange(n * next_n, dtype=torch.int32, device=dev).unsqueeze(1)
    assert torch.equal(gb.selected_attention(q, k, v, idx), v.repeat_interleave(heads // 2, 1))


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("next_n,q_heads,kv_heads,dim,n", [(1, 8, 2, 128, 20011), (9, 16, 2, 128, 9000), (17, 32, 2, 64, 5000),
                                                          (5, 12, 2, 256, 9000)])
@pytest.mark.parametrize("kind,gap,value", [("first", 24, 64), ("many", 20, 4), ("many", 44, 64)])
def test_tree_attention_with_a_sink_whose_score_is_zero(dev, dtype, next_n, q_heads, kv_heads, dim, n, kind, gap, value):
    """The others far below zero: the log-sum-exp is small, the references are
    not; and scores that are no whole powers of two."""
    g = torch.Generator(device=dev).manual_seed(gap + dim)
    at, zero = levels(kind, gap, n - next_n, g, dev)
    k = torch.zeros((n, kv_heads, dim), device=dev)
    k[:, :, 3] = -gap / 8
    k[:n - next_n, :, 3] += at.unsqueeze(1) / 8
    k[:, :, 5] = 0.01 * torch.randn((n, kv_heads), generator=g, device=dev)
    v = value * (1 + 0.25 * torch.randn(k.shape, generator=g, device=dev))
    v[:n - next_n][zero] = 0
    q = torch.zeros((next_n, q_heads, dim), device=dev)
    q[:, :, 3] = 8
    q[:, 1::2, 3] = 7
    q[:, :, 5] = torch.randn((next_n, q_heads), generator=g, device=dev)
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    table = torch.arange(n, dtype=torch.int32, device=dev).unsqueeze(0)
    out, lse = gb.tree_attention(q, k, v, table, torch.tensor([n], dtype=torch.int32, device=dev), next_n=next_n, scale=1.0,
                                 return_lse=True)
    group = q_heads // kv_heads
    for t in range(next_n):
        seen = n - next_n + t + 1
        for h in range(kv_heads):
            heads = slice(h * group, h * group + group)
            check(out[t, heads], lse[t, heads], q[t, heads], k[:seen, h], v[:seen, h], dtype)
