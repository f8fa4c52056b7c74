"""Writes into 4-bit caches at the ends of their range on the GPU: numbers beyond
the scales, of either sign and at every unit, and weights and frequencies that are
no numbers, against the formula in 64 bits, byte by byte."""
import math

import numpy as np
import pytest
import torch

import prefill_reference as ref
import sparse_attention_top_gb300 as gb

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def used_bytes(dim):
    c, s = ref.areas(dim)
    used = np.zeros(gb.int4_row_bytes(dim), dtype=bool)
    used[:dim // 2] = used[c:c + dim // 2] = used[2 * c:2 * c + dim // 16] = used[2 * c + s:2 * c + s + dim // 16] = True
    return used


def write(dev, k, v, freqs=None, positions=None, **kw):
    """The rows that k and v [tokens, heads, dim] become."""
    n, heads, dim = k.shape
    cache = torch.full((n, heads, gb.int4_row_bytes(dim)), 0xA5, dtype=torch.uint8, device=dev)
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    kw = {a: to(x) if isinstance(x, torch.Tensor) else x for a, x in kw.items()}
    gb.rotate_and_cache_int4(k.to(dev), k.to(dev), v.to(dev), to(positions), torch.arange(n, dtype=torch.int32, device=dev), to(freqs),
                             cache, **kw)
    return cache.cpu().numpy()[..., used_bytes(dim)]


def rows_of(yk, yv, k_unit, v_unit):
    dim = yk.shape[-1]
    return ref.row_bytes(*ref.codes(yk, k_unit), *ref.codes(yv, v_unit))[..., used_bytes(dim)]


def ends(dtype, dim):
    """Rows with infinities, NaN and the largest numbers of either sign."""
    most = 3e38 if dtype is BF else 65504.0
    x = torch.randn((8, 2, dim), generator=torch.Generator().manual_seed(dim)).to(dtype)
    x[0, :, 3], x[0, :, dim - 1] = -math.inf, math.inf
    x[1, :, 0], x[1, :, 1] = -most, most
    x[2, :, 2], x[2, :, 5] = math.nan, -most
    x[3, :] = -math.inf
    x[4, :, ::2] = -most
    x[5, :, 1::3] = -most / 4
    x[6, 0, 7] = -math.inf
    return x


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [32, 128, 256])
@pytest.mark.parametrize("log2_unit", [60, 9, 0, -8, -9, -12, -20, -60])
def test_signs_of_the_largest(dev, dtype, dim, log2_unit):
    """What lies beyond a scale's range is the largest code, of its own sign, at
    every unit; values, and keys as they are or rotated."""
    x, unit = ends(dtype, dim), 2.0 ** log2_unit
    got = write(dev, x, x, k_scale=unit, v_scale=unit)
    y = x.double().numpy()
    assert np.array_equal(got, rows_of(y, y, unit, unit))
    positions = torch.arange(8, dtype=torch.int32)
    freqs = (1.0 / (1 + torch.arange(dim // 4 // 8 * 8))).float()
    for pairs in (False, True):
        got = write(dev, x, x, freqs, positions, interleaved=pairs, k_scale=unit, v_scale=unit)
        with np.errstate(invalid="ignore"):
            turned, _ = ref.turned(y, positions.numpy(), freqs.numpy(), pairs, None, 0.0)
        assert np.array_equal(got, rows_of(turned, y, unit, unit))


@pytest.mark.parametrize("pairs", [False, True])
def test_weights_and_frequencies_that_are_no_numbers(dev, pairs):
    """A NaN is stored as 0, an infinity as the largest code, wherever it comes from."""
    dim = 64
    g = torch.Generator().manual_seed(5)
    k = torch.randn((5, 3, dim), generator=g).to(BF)
    w = torch.ones(dim)
    w[1], w[20], w[40], w[63] = math.nan, math.inf, -math.inf, 3e38
    freqs = torch.tensor([1.0, math.nan, 0.5, math.inf] + [0.1] * 4)
    positions = torch.tensor([0, 1, 7, -2, 900], dtype=torch.int32)
    kd, slots = k.to(dev), torch.arange(5, dtype=torch.int32, device=dev)
    for weight, inv in ((w, None), (None, freqs), (w, freqs)):
        cache = torch.zeros((5, 3, gb.int4_row_bytes(dim)), dtype=torch.uint8, device=dev)
        gb.rotate_and_cache_int4(kd, kd, kd, positions.to(dev), slots, None if inv is None else inv.to(dev), cache,
                                 k_weight=None if weight is None else weight.to(dev), interleaved=pairs)
        with np.errstate(invalid="ignore", over="ignore"):
            y, _ = ref.turned(k.double().numpy(), positions.numpy(), None if inv is None else inv.numpy(), pairs,
                              None if weight is None else weight.double().numpy(), float(np.float32(1e-6)))
        want = ref.row_bytes(*ref.codes(y), *ref.codes(k.double().numpy()))
        assert np.array_equal(cache.cpu().numpy()[..., used_bytes(dim)], want[..., used_bytes(dim)])
