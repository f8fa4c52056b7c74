"""Attention over 4-bit caches and packed prompts where scores are far from 0, on
the GPU: next to such scores a probability is 1 or 0, so each row's output is the
mean of the values at its largest score.  The scores are products of whole
numbers that 32 bits hold, times one factor: equal ones stay equal.

Tolerances, fixed beforehand: u |out| for the output's rounding, u sum p |v| for
the probabilities' and 2^-20 of it for the sums; lse relative to itself by
2^-21 (three roundings of the factor, one of the score, one of lse)."""
import math

import numpy as np
import pytest
import torch

import prefill_reference as ref
import sparse_attention_top_gb300 as gb

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}
# (scale of the scores, unit of a 4-bit cache's keys)
FACTORS = [(2.0 ** 16, 1.0), (-2.0 ** 27, 1.0), (2.0 ** 33, 1.0), (2.0 ** 102, 1.0), (-2.0 ** 108, 1.0), (1.7 * 2.0 ** 60, 2.0 ** 50),
           (2.0 ** -3, 2.0 ** 60), (3e3, 1.0)]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def check(out, lse, score, v, dtype, where):
    """out [dim], lse of a row whose seen scores are score [n] (as whole numbers and a factor), values v [n, dim]."""
    whole, factor = score
    top = (whole * factor).max()
    at = whole * factor == top
    o, mag = v[at].mean(0), np.abs(v[at]).mean(0)
    l = top + math.log(at.sum())
    tol = U[dtype] * np.abs(o) + (U[dtype] + 2.0 ** -20) * mag + (2.0 ** -25 if dtype is HF else 0)
    assert np.all(np.abs(out - o) <= tol), where
    assert abs(lse - l) <= 2.0 ** -21 * (1 + abs(l)), (where, lse, l)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("factor", FACTORS)
@pytest.mark.parametrize("heads,next_n,dim", [(4, 1, 64), (12, 1, 128), (8, 4, 64), (16, 4, 48), (3, 1, 256)])
@pytest.mark.parametrize("signs", ["all below", "both"])
def test_int4_scores_far_from_zero(dev, dtype, factor, heads, next_n, dim, signs):
    scale, unit = factor
    g = torch.Generator().manual_seed(dim + heads)
    lens = [700, 130, 9]
    slots = 840
    k = torch.randn((slots, 1, dim), generator=g)
    k[:, 0, 0] = torch.randint(1 if signs == "all below" else -7, 8, (slots,), generator=g).float()
    k[:, 0, 1:16] = 0
    k[:, 0, 1] = 7                    # (the block's scale is 1)
    v = torch.randn((slots, 1, dim), generator=g)
    rows = ref.row_bytes(*ref.codes(k.numpy()), *ref.codes(v.numpy()))
    kv, vv = ref.values(rows, dim)
    assert np.array_equal(kv[:, 0, 0], k[:, 0, 0].numpy())
    table = torch.randperm(slots, generator=g)[:sum(lens)].to(torch.int32)
    pages = torch.zeros((3, 700), dtype=torch.int32)
    for i, n in enumerate(lens):
        pages[i, :n] = table[sum(lens[:i]):sum(lens[:i]) + n]
    q = torch.zeros((3 * next_n, heads, dim))
    q[:, :, 0] = torch.randint(1, 4, (3 * next_n, heads), generator=g) * (-1.0 if (scale > 0) == (signs == "all below") else 1.0)
    out, lse = gb.tree_attention_int4(q.to(dtype).to(dev), torch.from_numpy(rows).to(dev), pages.to(dev),
                                      torch.tensor(lens, dtype=torch.int32, device=dev), next_n=next_n, scale=scale, k_scale=unit,
                                      return_lse=True)
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    for r in range(3 * next_n):
        i, t = divmod(r, next_n)
        seen = pages[i, :lens[i] - next_n + t + 1].long().numpy()
        for h in range(heads):
            check(out[r, h], lse[r, h], (kv[seen, 0, 0] * float(q[r, h, 0]), scale * unit), vv[seen, 0], dtype, (r, h))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("scale", [f for f, unit in FACTORS if unit == 1.0])
@pytest.mark.parametrize("heads,kv,dim", [(4, 2, 64), (2, 2, 128), (3, 1, 256)])
@pytest.mark.parametrize("signs", ["all below", "both"])
def test_prompt_scores_far_from_zero(dev, dtype, scale, heads, kv, dim, signs):
    g = torch.Generator().manual_seed(dim + heads)
    lens = [400, 1, 130]
    n = sum(lens)
    k = torch.zeros((n, kv, dim))
    k[:, :, 0] = torch.randint(1 if signs == "all below" else -7, 8, (n, kv), generator=g).float()
    v = torch.randn((n, kv, dim), generator=g).to(dtype)
    q = torch.randn((n, heads, dim), generator=g) * 0
    q[:, :, 0] = torch.randint(1, 4, (n, heads), generator=g) * (-1.0 if (scale > 0) == (signs == "all below") else 1.0)
    cu = np.cumsum([0] + lens)
    out, lse = gb.prompt_attention(q.to(dtype).to(dev), k.to(dtype).to(dev), v.to(dev), torch.from_numpy(cu).to(torch.int32).to(dev),
                                   scale=scale, return_lse=True)
    out, lse, kk, vv = out.cpu().double().numpy(), lse.cpu().double().numpy(), k.double().numpy(), v.double().numpy()
    for i in range(3):
        for t in list(range(0, lens[i], 37)) + [lens[i] - 1]:
            r, seen = cu[i] + t, slice(cu[i], cu[i] + t + 1)
            for h in range(heads):
                c = h // (heads // kv)
                check(out[r, h], lse[r, h], (kk[seen, c, 0] * float(q[r, h, 0]), scale), vv[seen, c], dtype, (i, t, h))
