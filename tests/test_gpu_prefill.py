"""Norms, rotation and cache writes on the GPU against their definitions in 64
bits.

Tolerances, fixed beforehand: an element that is rounded to a 16-bit type may
be off by half a step of it (u |y|, and half of the smallest subnormal) plus
2^-19 of the magnitudes it is a sum of: in units of 2^-24 the sum of squares is
off by 14 relative to itself (halved by the root), the root by 4, three
products by 1 each, cosine and sine by 4 and by the rounding of the turns, pi;
32 is more than their sum.  Values and 4-bit codes are exact."""
import math

import numpy as np
import pytest
import torch

import decode_reference as dref
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


class Tokens:
    def __init__(self, rows, q_heads, kv, dim, freqs, dtype, seed, norm=True, wide_weights=False, far=1000, fused=True):
        g = torch.Generator().manual_seed(seed)
        width = q_heads + 2 * kv
        both = torch.randn((rows, width, dim), generator=g).to(dtype)
        self.both, self.q_heads, self.kv, self.dim, self.dtype, self.fused = both, q_heads, kv, dim, dtype, fused
        self.positions = torch.randint(-5, far, (rows,), generator=g, dtype=torch.int32)
        self.freqs = (1e4 ** (-torch.arange(freqs, dtype=torch.float64) / max(1, freqs))).float() if freqs else None
        self.slots = torch.randperm(rows + 9, generator=g)[:rows].to(torch.int32)
        self.num_slots = rows + 9
        wt = torch.float32 if wide_weights else dtype
        self.wq, self.wk = ((1 + 0.2 * torch.randn((2, dim), generator=g)).to(wt) if norm else (None, None))

    def parts(self, dev):
        b = self.both.to(dev)
        h = self.q_heads
        got = [b[:, :h], b[:, h:h + self.kv], b[:, h + self.kv:]]
        return got if self.fused else [x.contiguous() for x in got]

    def args(self, dev):
        to = lambda t: None if t is None else t.to(dev)  # noqa: E731
        return (self.positions.to(dev), self.slots.to(dev), to(self.freqs)), dict(q_weight=to(self.wq), k_weight=to(self.wk))

    def expect(self, interleaved, eps):
        h = self.q_heads
        x = self.both.double().numpy()
        f = None if self.freqs is None else self.freqs.numpy()
        pos = self.positions.numpy()
        w = [None if t is None else t.double().numpy() for t in (self.wq, self.wk)]
        return (ref.turned(x[:, :h], pos, f, interleaved, w[0], eps), ref.turned(x[:, h:h + self.kv], pos, f, interleaved, w[1], eps),
                x[:, h + self.kv:])


def near(got, y, mag, dtype):
    got = got.cpu().double().numpy()
    tol = U[dtype] * (np.abs(y) + 2.0 ** -19 * mag) + 2.0 ** -19 * mag + SMALL[dtype]
    assert np.all(np.abs(got - y) <= tol), np.max(np.abs(got - y) - tol)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,q_heads,kv,dim,freqs,kw", [
    (1, 1, 1, 8, 0, {}),
    (1, 32, 8, 128, 64, {}),
    (5, 6, 2, 64, 32, dict(norm=False)),
    (33, 7, 7, 80, 40, dict(wide_weights=True)),
    (17, 16, 1, 256, 128, dict(fused=False)),
    (3, 40, 20, 72, 16, dict(far=1 << 20)),
    (700, 4, 2, 192, 96, dict(far=1 << 20)),
    (40, 12, 4, 96, 0, dict(wide_weights=True)),
])
def test_rotate_and_cache(dev, dtype, interleaved, rows, q_heads, kv, dim, freqs, kw):
    t = Tokens(rows, q_heads, kv, dim, freqs, dtype, rows + dim, **kw)
    t.slots[rows // 2] = -1 if rows > 1 else t.slots[0]
    if rows > 4:
        t.slots[1] = t.num_slots          # behind the cache: not written
    fill = torch.full((t.num_slots, 2, kv, dim), 3.5, dtype=dtype, device=dev)
    kc, vc = fill[:, 0], fill[:, 1]
    q, k, v = t.parts(dev)
    args, w = t.args(dev)
    out = gb.rotate_and_cache(q, k, v, *args, kc, vc, interleaved=interleaved, eps=1e-5, **w)
    (yq, mq), (yk, mk), yv = t.expect(interleaved, 1e-5)
    near(out, yq, mq, dtype)
    there = [i for i, s in enumerate(t.slots.tolist()) if 0 <= s < t.num_slots]
    at = t.slots[there].long().to(dev)
    near(kc[at], yk[there], mk[there], dtype)
    assert np.array_equal(vc[at].cpu().double().numpy(), yv[there])
    rest = torch.ones(t.num_slots, dtype=torch.bool)
    rest[at.cpu()] = False
    assert bool((fill[rest.to(dev)] == 3.5).all())          # no other slot is touched
    # in place
    again = gb.rotate_and_cache(q, k, v, *args, kc, vc, interleaved=interleaved, eps=1e-5, q_out=q, **w)
    assert again is q and torch.equal(q, out)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,q_heads,kv,dim,freqs,kw", [
    (1, 8, 8, 16, 8, {}),
    (5, 6, 2, 64, 32, dict(norm=False)),
    (33, 7, 7, 80, 40, dict(wide_weights=True)),
    (17, 16, 1, 256, 64, {}),
    (9, 4, 4, 112, 56, dict(far=1 << 20)),
    (1500, 4, 4, 128, 64, dict(far=1 << 20)),
    (64, 2, 2, 192, 0, dict(norm=False)),
])
def test_rotate_and_cache_int4(dev, dtype, interleaved, rows, q_heads, kv, dim, freqs, kw):
    """Every byte is the formula's; what is read back is its values."""
    t = Tokens(rows, q_heads, kv, dim, freqs, dtype, rows * 3 + dim, **kw)
    # blocks of many magnitudes, so that scales of every binade come up
    g = torch.Generator().manual_seed(dim)
    size = torch.exp2(torch.randint(-12, 13, (rows, t.both.shape[1], dim // 16, 1), generator=g).float())
    if t.wk is None:
        t.both = (t.both.view(rows, -1, dim // 16, 16) * size).view(rows, -1, dim).to(dtype)
    if rows > 4:
        t.slots[1], t.slots[3] = -1, t.num_slots
    n = gb.int4_row_bytes(dim)
    big = torch.full((t.num_slots, kv, n + 16), 0xA5, dtype=torch.uint8, device=dev)
    cache = big[:, :, :n]
    q, k, v = t.parts(dev)
    args, w = t.args(dev)
    k_unit, v_unit = (1.0, 1.0) if dim != 80 else (0.25, 2.0)
    out = gb.rotate_and_cache_int4(q, k, v, *args, cache, interleaved=interleaved, k_scale=k_unit, v_scale=v_unit, **w)
    (yq, mq), (yk, _), yv = t.expect(interleaved, float(np.float32(1e-6)))
    near(out, yq, mq, dtype)
    there = [i for i, s in enumerate(t.slots.tolist()) if 0 <= s < t.num_slots]
    at = t.slots[there].long().to(dev)
    want = ref.row_bytes(*ref.codes(yk[there], k_unit), *ref.codes(yv[there], v_unit))
    got = cache[at].cpu().numpy()
    c, s = ref.areas(dim)
    used = np.zeros(n, dtype=bool)
    used[:dim // 2] = used[c:c + dim // 2] = used[2 * c:2 * c + dim // 16] = used[2 * c + s:2 * c + s + dim // 16] = True
    assert np.array_equal(got[..., used], want[..., used])
    rest = torch.ones(t.num_slots, dtype=torch.bool)
    rest[at.cpu()] = False
    assert bool((big[rest.to(dev)] == 0xA5).all()) and bool((big[:, :, n:] == 0xA5).all())
    # read back, with slots that do not exist
    slots = t.slots.to(dev)
    rk, rv = gb.read_cache_int4(cache, slots, dim, dtype, k_scale=k_unit, v_scale=v_unit)
    wk, wv = np.zeros((rows, kv, dim)), np.zeros((rows, kv, dim))
    a, b = ref.values(got, dim)
    wk[there], wv[there] = a * k_unit, b * v_unit
    assert torch.equal(rk.cpu(), torch.from_numpy(wk).to(dtype)) and torch.equal(rv.cpu(), torch.from_numpy(wv).to(dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [16, 48, 128, 256])
def test_read_every_byte(dev, dtype, dim):
    """Rows of random bytes: every code and scale pattern, the ones no write
    makes included, is a number."""
    g = torch.Generator().manual_seed(dim)
    n = gb.int4_row_bytes(dim)
    cache = torch.randint(0, 256, (500, 3, n), generator=g, dtype=torch.uint8)
    slots = torch.randint(-3, 510, (2000,), generator=g, dtype=torch.int32)
    k, v = gb.read_cache_int4(cache.to(dev), slots.to(dev), dim, dtype)
    a, b = ref.values(cache.numpy(), dim)
    ok = ((slots >= 0) & (slots < 500)).numpy()
    for got, x in ((k, a), (v, b)):
        want = np.where(ok[:, None, None], x[slots.clamp(0, 499).numpy()], 0.0)
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(dtype))
    e = gb.read_cache_int4(cache.to(dev), slots[:0].to(dev), dim, dtype)
    assert e.k.shape == (0, 3, dim)


def test_int4_ends(dev):
    """Zeros, infinities, NaN, numbers below and beyond the scales."""
    dim = 64
    rows = torch.zeros((6, 3, dim), dtype=BF)
    rows[1] = 3e38
    rows[2] = 1e-30
    rows[3, :, 5], rows[3, :, 20], rows[3, :, 33] = math.inf, -math.inf, math.nan
    rows[3, :, 40] = 2.0
    rows[4] = torch.linspace(-4000, 4000, dim)
    rows[5] = torch.arange(dim) * 2.0 ** -12
    q, k, v = (rows[:, i:i + 1].contiguous().to(dev) for i in range(3))
    slots = torch.arange(6, dtype=torch.int32, device=dev)
    cache = torch.zeros((6, 1, gb.int4_row_bytes(dim)), dtype=torch.uint8, device=dev)
    gb.rotate_and_cache_int4(q, k, v, None, slots, None, cache)
    x = rows[:, 0].double().numpy()
    want = ref.row_bytes(*ref.codes(x), *ref.codes(x))
    assert np.array_equal(cache[:, 0].cpu().numpy(), want)
    k, v = gb.read_cache_int4(cache, slots, dim)
    assert bool(torch.isfinite(k).all() and torch.isfinite(v).all()) and float(k[1, 0, 0]) == 7 * 448


def test_padded_batch_replays(dev):
    """A captured write with slots, positions and inputs that change between
    replays; padding tokens come and go."""
    t = Tokens(24, 8, 2, 128, 64, BF, 5)
    q, k, v = (x.contiguous() for x in t.parts(dev))
    (pos, slots, freq), w = t.args(dev)
    cache = torch.zeros((t.num_slots, 2, gb.int4_row_bytes(128)), dtype=torch.uint8, device=dev)
    out = torch.empty_like(q)

    def call():
        gb.rotate_and_cache_int4(q, k, v, pos, slots, freq, cache, q_out=out, **w)
        return gb.read_cache_int4(cache, slots, 128)

    call()
    torch.cuda.synchronize(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(BF))
        pos.copy_(torch.randint(0, 9999, (24,), generator=g, dtype=torch.int32))
        s = torch.randperm(t.num_slots, generator=g)[:24].to(torch.int32)
        s[20 - seed:] = -1
        slots.copy_(s)
        cache.zero_()
        graph.replay()
        torch.cuda.synchronize(dev)
        kept, out_kept = [x.clone() for x in got], out.clone()
        cache.zero_()
        eager = call()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager)) and torch.equal(out, out_kept)
        assert bool((kept[0][20 - seed:] == 0).all()) and bool((kept[0][0] != 0).any())


def test_rotate_refuses(dev):
    t = Tokens(4, 4, 2, 64, 32, BF, 1)
    q, k, v = t.parts(dev)
    (pos, slots, freq), w = t.args(dev)
    kc = torch.zeros((t.num_slots, 2, 64), dtype=BF, device=dev)
    c4 = torch.zeros((t.num_slots, 2, gb.int4_row_bytes(64)), dtype=torch.uint8, device=dev)

    def call(**kw):
        a = dict(q=q, k=k, v=v, positions=pos, slots=slots, inv_freq=freq, k_cache=kc, v_cache=kc.clone(), **w)
        a.update(kw)
        return gb.rotate_and_cache(**a)

    def call4(**kw):
        a = dict(q=q, k=k, v=v, positions=pos, slots=slots, inv_freq=freq, cache=c4, **w)
        a.update(kw)
        return gb.rotate_and_cache_int4(**a)

    call(), call4()
    for bad in (dict(q=q.float()), dict(k=k[:3]), dict(k=k.half()), dict(v=v[:, :1]), dict(slots=slots.long()),
                dict(slots=slots[:3]), dict(positions=pos[:2]), dict(inv_freq=freq[:12]), dict(inv_freq=freq.double()),
                dict(inv_freq=torch.cat([freq, freq])), dict(q_weight=w["q_weight"].half()), dict(k_weight=w["k_weight"][:32]),
                dict(k_weight=w["k_weight"].float()), dict(eps=-1.0), dict(q_out=q[:2]), dict(q=q.transpose(1, 2)),
                dict(positions=None), dict(q=q[:, :3]), dict(q=q.cpu())):
        for f in (call, call4):
            with pytest.raises(ValueError):
                f(**bad)
    for bad in (dict(k_cache=kc[:, :1]), dict(v_cache=kc[:3]), dict(k_cache=kc.half())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(cache=c4[..., :64]), dict(cache=c4.to(torch.int8)), dict(cache=c4[:, :1]), dict(k_scale=0.3),
                dict(v_scale=0.0), dict(v_scale=-1.0), dict(k_scale=math.inf), dict(k_scale=math.nan)):
        with pytest.raises(ValueError):
            call4(**bad)
    for bad in (dict(slots=slots.long()), dict(dtype=torch.float32), dict(head_dim=60), dict(head_dim=128), dict(k_scale=3.0),
                dict(k_out=kc)):
        a = dict(cache=c4, slots=slots, head_dim=64)
        a.update(bad)
        with pytest.raises(ValueError):
            gb.read_cache_int4(**a)
