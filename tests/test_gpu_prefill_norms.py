"""Norms at the ends of their range on the GPU: rows whose sum of squares is more
or less than 32 bits hold, beside ordinary ones, against the formula in 64 bits.
4-bit codes are exact; rounded elements have the tolerances of
test_gpu_prefill.py, of which the root and the sum are then better than they
have to be."""
import math

import numpy as np
import pytest
import torch

import prefill_reference as ref
import sparse_attention_top_gb300 as gb

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}
SMALL = {BF: 2.0 ** -134, HF: 2.0 ** -25}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def near(got, y, mag, dtype):
    got = got.cpu().double().numpy()
    tol = U[dtype] * (np.abs(y) + 2.0 ** -19 * mag) + 2.0 ** -19 * mag + SMALL[dtype]
    nan = np.isnan(y)
    assert np.array_equal(nan, np.isnan(got))
    assert np.all(np.abs(got - y)[~nan] <= tol[~nan]), np.max(np.abs(got - y)[~nan] - tol[~nan])


def used_bytes(dim):
    c, s = ref.areas(dim)
    used = np.zeros(gb.int4_row_bytes(dim), dtype=bool)
    used[:dim // 2] = used[c:c + dim // 2] = used[2 * c:2 * c + dim // 16] = used[2 * c + s:2 * c + s + dim // 16] = True
    return used


SIZES = [1e20, 1.0, 3e37, 2e18, 1e-12, 1e-19, 1e-25, 1e-38]


def sized(tokens, heads, dim, seed):
    """Rows of many sizes, none alike its neighbours'; every fifth with one element that is all of it."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, heads, dim), generator=g).clamp(-4, 4).double()
    at = torch.arange(tokens * heads).view(tokens, heads)
    x = x * torch.tensor(SIZES, dtype=torch.float64)[(at + tokens // 3) % len(SIZES)].unsqueeze(2)
    one = at % 5 == 4
    x[one] *= 2.0 ** -60
    x[:, :, dim // 3][one] = torch.tensor(SIZES, dtype=torch.float64)[at[one] % len(SIZES)]
    return x.to(BF)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,freqs", [(1, 1, 16, 0), (19, 5, 64, 32), (9, 4, 128, 32), (3, 3, 256, 128), (700, 2, 80, 40)])
@pytest.mark.parametrize("weights", [True, False])
def test_norms_of_rows_of_any_size(dev, eps, interleaved, tokens, heads, dim, freqs, weights):
    q, k, v = (sized(tokens, heads, dim, s) for s in (1, 2, 3))
    g = torch.Generator().manual_seed(4)
    wq, wk = (1 + 0.2 * torch.randn((2, dim), generator=g) if weights else torch.ones((2, dim))).to(BF)
    positions = torch.randint(0, 4000, (tokens,), generator=g, dtype=torch.int32)
    inv = (1e4 ** (-torch.arange(freqs, dtype=torch.float64) / max(1, freqs))).float() if freqs else None
    slots = torch.randperm(tokens, generator=g).to(torch.int32)
    args = [positions.to(dev), slots.to(dev), None if inv is None else inv.to(dev)]
    how = dict(q_weight=wq.to(dev), k_weight=wk.to(dev), eps=eps, interleaved=interleaved)
    turned = lambda x, w: ref.turned(x.double().numpy(), positions.numpy(), None if inv is None else inv.numpy(), interleaved,  # noqa: E731
                                     w.double().numpy(), float(np.float32(eps)))
    (yq, mq), (yk, mk) = turned(q, wq), turned(k, wk)
    at = slots.long().numpy()
    kc, vc = torch.zeros((2, tokens, heads, dim), dtype=BF, device=dev)
    qd, kd, vd = q.to(dev), k.to(dev), v.to(dev)
    out = gb.rotate_and_cache(qd, kd, vd, *args, kc, vc, **how)
    near(out, yq, mq, BF)
    near(kc[slots.long().to(dev)], yk, mk, BF)
    cache = torch.zeros((tokens, heads, gb.int4_row_bytes(dim)), dtype=torch.uint8, device=dev)
    # in place
    assert gb.rotate_and_cache_int4(qd, kd, vd, *args, cache, q_out=qd, **how) is qd and torch.equal(qd, out)
    want = ref.row_bytes(*ref.codes(yk), *ref.codes(v.double().numpy()))
    used = used_bytes(dim)
    assert np.array_equal(cache.cpu().numpy()[at][..., used], want[..., used])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_without_a_norm(dev, dtype, dim):
    """Rows with an infinity or NaN beside ordinary ones and ones of the largest numbers."""
    g = torch.Generator().manual_seed(dim)
    x = torch.randn((6, 4, dim), generator=g).to(dtype)
    x[0, 1, 5], x[1, 0, 0], x[2, 3, dim - 1] = math.nan, math.inf, -math.inf
    x[3, 2] = (torch.randn(dim, generator=g).clamp(-3, 3) * (1e38 if dtype is BF else 2e4)).to(dtype)
    w = torch.ones(dim, dtype=dtype)
    slots = torch.arange(6, dtype=torch.int32, device=dev)
    kc, vc = torch.zeros((2, 6, 4, dim), dtype=dtype, device=dev)
    xd = x.to(dev)
    out = gb.rotate_and_cache(xd, xd, xd, None, slots, None, kc, vc, q_weight=w.to(dev), k_weight=w.to(dev))
    with np.errstate(invalid="ignore"):
        y, mag = ref.turned(x.double().numpy(), None, None, False, w.double().numpy(), float(np.float32(1e-6)))
    near(out, y, mag, dtype)
    near(kc, y, mag, dtype)
    cache = torch.zeros((6, 4, gb.int4_row_bytes(dim)), dtype=torch.uint8, device=dev)
    gb.rotate_and_cache_int4(xd, xd, xd, None, slots, None, cache, k_weight=w.to(dev))
    want = ref.row_bytes(*ref.codes(y), *ref.codes(x.double().numpy()))
    used = used_bytes(dim)
    assert np.array_equal(cache.cpu().numpy()[..., used], want[..., used])
