"""Attention over packed prompts on the GPU against its definition in 64 bits.

Tolerances, fixed beforehand: u |out| for the output's own rounding and (u + 2
eta) sum p |v|, with eta the bound on a score's error and u what a probability
is rounded by; lse by eta and 32-bit rounding (as for the cached attention)."""
import math

import numpy as np
import pytest
import torch

import prefill_reference as ref
import sparse_attention_top_gb300 as gb

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


class Packed:
    """Sequences one behind another; what no sequence owns is NaN."""

    def __init__(self, lens, klens, q_heads, kv, dim, dtype, seed, gap=0, tail=3, fused=False):
        g = torch.Generator().manual_seed(seed)
        klens = lens if klens is None else klens
        self.cu = np.cumsum([gap] + lens).astype(np.int32)
        self.cuk = np.cumsum([gap] + klens).astype(np.int32)
        rows, keys = int(self.cu[-1]) + tail, int(self.cuk[-1]) + tail
        self.q = torch.randn((rows, q_heads, dim), generator=g).to(dtype)
        kv_t = torch.randn((keys, 2 * kv, dim) if fused else (2, keys, kv, dim), generator=g).to(dtype)
        self.k, self.v = (kv_t[:, :kv], kv_t[:, kv:]) if fused else (kv_t[0], kv_t[1])
        for t, cu in ((self.q, self.cu), (self.k, self.cuk), (self.v, self.cuk)):
            t[:gap], t[int(cu[-1]):] = math.nan, math.nan
        self.dtype, self.group, self.scale = dtype, q_heads // kv, dim ** -0.5

    def call(self, dev, **kw):
        same = np.array_equal(self.cu, self.cuk)
        k, v = (self.k.to(dev), self.v.to(dev))
        if self.k.stride(0) != self.k.shape[1] * self.k.shape[2]:      # parts of one tensor
            both = torch.cat([self.k, self.v], 1).to(dev)
            k, v = both[:, :self.k.shape[1]], both[:, self.k.shape[1]:]
        return gb.prompt_attention(self.q.to(dev), k, v, torch.from_numpy(self.cu).to(dev),
                                   cu_seqlens_k=None if same else torch.from_numpy(self.cuk).to(dev), return_lse=True, **kw)

    def check(self, out, lse, rows=None, scale=None):
        q, k, v = (x.double().numpy() for x in (self.q, self.k, self.v))
        scale = self.scale if scale is None else scale
        out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
        for i in range(len(self.cu) - 1):
            n, m = int(self.cu[i + 1] - self.cu[i]), int(self.cuk[i + 1] - self.cuk[i])
            for t in range(n) if rows is None else [t for t in rows if t < n]:
                r, seen = int(self.cu[i]) + t, max(0, m - n + t + 1)
                at = slice(int(self.cuk[i]), int(self.cuk[i]) + seen)
                o, l, eta, mag = ref.attend(q[r], k[at] if scale >= 0 else -k[at], v[at], self.group, abs(scale))
                tol = U[self.dtype] * np.abs(o) + (U[self.dtype] + 2 * eta[:, None]) * mag + (2.0 ** -25 if self.dtype is HF else 0)
                assert not (np.abs(out[r] - o) > tol).any(), (i, t, np.max(np.abs(out[r] - o) - tol))
                none = l == -math.inf
                assert np.array_equal(none, lse[r] == -math.inf)
                assert np.all(np.abs(lse[r][~none] - l[~none]) <= eta[~none] + 2.0 ** -21 * (1 + np.abs(l[~none]))), (i, t)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,klens,q_heads,kv,dim", [
    ([1], None, 1, 1, 64),
    ([1, 2, 3, 0, 5], None, 4, 2, 128),
    ([130, 127, 128, 129, 300], None, 2, 2, 128),        # one head a group: 256 tokens a unit
    ([70, 0, 33, 257], None, 8, 1, 64),                  # eight heads a group
    ([40, 513], None, 12, 2, 80),                        # six: three times two
    ([65, 31], None, 7, 1, 96),                          # seven: each head by itself
    ([200, 129], None, 4, 4, 256),
    ([90, 300], None, 8, 2, 136),
    ([33], None, 16, 16, 8),
    ([17, 260], None, 128, 1, 72),                       # a token's heads fill a row tile
    ([5, 100, 1], [700, 100, 129], 4, 1, 128),           # chunks behind their context
    ([100, 4, 260, 7], [30, 0, 200, 7], 4, 2, 64),       # rows that see nothing
    ([100, 260], [30, 200], 2, 2, 192),
])
def test_prompt_attention(dev, dtype, lens, klens, q_heads, kv, dim):
    b = Packed(lens, klens, q_heads, kv, dim, dtype, seed=sum(lens) + dim, gap=len(lens) % 3, fused=dim in (64, 96, 256))
    out = torch.full(b.q.shape, 7.0, dtype=dtype, device=dev)
    lse = torch.full(b.q.shape[:2], 7.0, device=dev)
    got = b.call(dev, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    b.check(out, lse)
    first, end = int(b.cu[0]), int(b.cu[-1])
    for t in (out, lse):                                 # rows of no sequence stay
        assert bool((t[:first] == 7).all()) and bool((t[end:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 4.0])
def test_scales(dev, dtype, scale):
    b = Packed([150, 40], None, 4, 2, 64, dtype, seed=3)
    b.check(*b.call(dev, scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("q_heads,kv,dim", [(2, 1, 64), (1, 1, 128), (4, 4, 256)])
def test_long_and_many(dev, dtype, q_heads, kv, dim):
    """Many units a block, long rows, references that move: sampled rows."""
    b = Packed([5000] + [61] * 60 + [1800], None, q_heads, kv, dim, dtype, seed=dim, tail=100)
    at = torch.arange(b.k.shape[0]).view(-1, 1, 1)
    b.k = (b.k.float() * (0.3 + at / 3000.0)).to(dtype)
    out, lse = b.call(dev)
    b.check(out, lse, rows=[0, 1, 60, 127, 128, 255, 1023, 1799, 2500, 4095, 4999])
    again = b.call(dev)
    end = int(b.cu[-1])
    assert torch.equal(out[:end], again[0][:end]) and torch.equal(lse[:end], again[1][:end])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("q_heads,kv,dim", [(4, 2, 128), (2, 2, 64), (3, 1, 256)])
def test_infinities_and_nan_stay_with_rows_that_see_them(dev, dtype, q_heads, kv, dim):
    b = Packed([300, 200, 64], None, q_heads, kv, dim, dtype, seed=8)
    bad = {(0, 130): math.nan, (0, 299): math.inf, (1, 0): None, (1, 77): -math.inf, (1, 199): math.nan, (2, 63): math.inf}
    clean_v = b.v.clone()
    for (i, t), x in bad.items():
        if x is not None:
            b.v[int(b.cu[i]) + t, 0, 5 % dim] = x
    b.k[int(b.cu[0]) + 250, 0, 1] = math.nan             # a key: its scores are NaN for the rows that see it
    out, lse = b.call(dev)
    out, lse = out.cpu(), lse.cpu()
    heads = slice(0, b.group)                            # of kv head 0
    for i, n in enumerate([300, 200, 64]):
        o = out[int(b.cu[i]):int(b.cu[i + 1])]
        first = min([t for (j, t), x in bad.items() if j == i and x is not None])
        assert bool(torch.isfinite(o[:first]).all())
        other = [d for d in range(dim) if d != 5 % dim]
        upto = 250 if i == 0 else n
        assert not bool(torch.isfinite(o[first:, heads, 5 % dim]).any())
        assert bool(torch.isfinite(o[:upto, heads][:, :, other]).all())
        if kv > 1:
            assert bool(torch.isfinite(o[:, b.group:]).all())
    assert bool(torch.isnan(out[250:300, heads]).all()) and bool(torch.isnan(lse[250:300, heads]).all())
    assert float(out[int(b.cu[1]) + 80, 0, 5 % dim]) == -math.inf
    # what is finite is right: rows before the first bad one, and the other heads
    b.v = clean_v
    b.k[int(b.cu[0]) + 250, 0, 1] = 0.0
    good = Packed([130, 77, 63], None, q_heads, kv, dim, dtype, seed=1)
    for name in "qkv":
        src, dst = getattr(b, name), getattr(good, name)
        for i in range(3):
            n = int(good.cu[i + 1] - good.cu[i])
            dst[int(good.cu[i]):int(good.cu[i + 1])] = src[int(b.cu[i]):int(b.cu[i]) + n]
    where = torch.cat([torch.arange(int(b.cu[i]), int(b.cu[i]) + int(good.cu[i + 1] - good.cu[i])) for i in range(3)])
    good.check(out[where], lse[where])


def test_offsets_that_are_not_ascending(dev):
    """They are clamped: nothing is read or written out of place."""
    b = Packed([100, 100], None, 4, 2, 64, BF, seed=5, tail=0)
    cu = torch.tensor([50, 20, 9999, -7, 200, 0, 200], dtype=torch.int32, device=dev)
    big = torch.full((300, 4, 64), 7.0, dtype=BF, device=dev)
    ws = torch.zeros(gb.gbtopk_prompt_workspace_bytes(200, 6, 4, 2, 64) + 4096, dtype=torch.uint8, device=dev)
    n = gb.gbtopk_prompt_workspace_bytes(200, 6, 4, 2, 64)
    ws[n:] = 0xA5
    gb.prompt_attention(b.q.to(dev), b.k.to(dev), b.v.to(dev), cu, out=big[50:250], workspace=ws[:n])
    torch.cuda.synchronize(dev)
    assert bool((big[:50] == 7).all()) and bool((big[250:] == 7).all()) and bool((ws[n:] == 0xA5).all())
    assert gb.gbtopk_device_status(ws[:n]) == 0


def test_replays_other_lengths_on_another_stream(dev):
    b = Packed([200, 90, 110], None, 4, 2, 128, HF, seed=6, tail=60)
    stream = torch.cuda.Stream(dev)
    q, k, v = b.q.to(dev), b.k.to(dev), b.v.to(dev)
    q, k, v = (torch.nan_to_num(x, 0.5) for x in (q, k, v))
    b.q, b.k, b.v = q.cpu(), k.cpu(), v.cpu()
    cu = torch.from_numpy(b.cu).to(dev)
    torch.cuda.synchronize(dev)
    with torch.cuda.stream(stream):
        gb.prompt_attention(q, k, v, cu)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = gb.prompt_attention(q, k, v, cu, return_lse=True)
    for lens in ([1, 0, 350], [0, 0, 0], [130, 200, 130]):
        new = np.cumsum([0] + lens).astype(np.int32)
        cu.copy_(torch.from_numpy(new))
        torch.cuda.synchronize(dev)
        graph.replay()
        torch.cuda.synchronize(dev)
        b.cu = b.cuk = new
        b.check(*got)


def test_empty_calls(dev):
    z = torch.zeros((0, 4, 64), dtype=BF, device=dev)
    one = torch.zeros((3, 4, 64), dtype=BF, device=dev)
    cu = torch.zeros(1, dtype=torch.int32, device=dev)
    assert gb.prompt_attention(z, z[:, :2], z[:, :2], cu).shape == (0, 4, 64)
    assert gb.prompt_attention(one, one[:, :2], one[:, :2], cu).shape == (3, 4, 64)
    two = torch.tensor([0, 3], dtype=torch.int32, device=dev)
    out, lse = gb.prompt_attention(one, z[:, :2], z[:, :2], two, cu_seqlens_k=torch.zeros(2, dtype=torch.int32, device=dev), return_lse=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_prompt_attention_refuses(dev):
    b = Packed([20, 10], None, 4, 2, 64, BF, seed=1)
    q, k, v, cu = b.q.to(dev), b.k.to(dev), b.v.to(dev), torch.from_numpy(b.cu).to(dev)

    def call(**kw):
        a = dict(q=q, k=k, v=v, cu_seqlens=cu)
        a.update(kw)
        return gb.prompt_attention(**a)
    call()
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(v=v[:5]), dict(k=k[:, :1]), dict(q=q[:, :3]), dict(q=q[..., :32]),
                dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu[:0]), dict(cu_seqlens_k=cu[:2]), dict(cu_seqlens_k=cu.float()),
                dict(out=q[:3]), dict(lse=torch.zeros(3, device=dev)), dict(workspace=torch.zeros(16, dtype=torch.uint8, device=dev)),
                dict(q=q.cpu()), dict(k=k[:, :1].expand(-1, 2, -1), v=v[:, :1].expand(-1, 2, -1))):
        with pytest.raises(ValueError):
            call(**bad)
