"""Layouts of queries, keys, values and caches that the prompt's calls document and
their other tests do not have: heads outermost, rows padded to odd multiples of 8
elements, every other head or slot of a larger tensor.  Strides move no number: the
results are those of dense copies, to the bit."""
import pytest
import torch

import sparse_attention_top_gb300 as gb

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def heads_first(x):
    return x.transpose(0, 1).contiguous().transpose(0, 1)


def padded(x, rows, heads):
    """Rows `rows` elements longer than they have to be, heads `heads`."""
    n, h, d = x.shape
    row = h * (d + heads) + rows
    big = torch.full((n * row + 64,), 3.0, dtype=x.dtype, device=x.device)
    view = big.as_strided((n, h, d), (row, d + heads, 1), 8)
    view.copy_(x)
    return view


def every_other(x):
    n, h, d = x.shape
    big = torch.full((2 * n, 3 * h, d), 3.0, dtype=x.dtype, device=x.device)
    view = big[::2, 1::3]
    view.copy_(x)
    return view


LAYOUTS = {"heads first": heads_first, "rows padded": lambda x: padded(x, 8, 0), "heads padded": lambda x: padded(x, 40, 24),
           "every other": every_other}


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("q_heads,kv,dim", [(8, 2, 128), (6, 6, 40), (12, 1, 64), (4, 2, 256)])
def test_prompt_attention(dev, layout, dtype, q_heads, kv, dim):
    g = torch.Generator().manual_seed(dim)
    n = 330
    q, k, v = (torch.randn((n, h, dim), generator=g).to(dtype).to(dev) for h in (q_heads, kv, kv))
    cu = torch.tensor([0, 130, 131, n], dtype=torch.int32, device=dev)
    want = gb.prompt_attention(q, k, v, cu, return_lse=True)
    f = LAYOUTS[layout]
    got = gb.prompt_attention(f(q), f(k), f(v), cu, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    mixed = gb.prompt_attention(q, f(k), LAYOUTS["rows padded"](v), cu, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(mixed, want))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("q_heads,kv,dim,freqs", [(8, 2, 128, 64), (6, 6, 48, 16), (4, 2, 256, 96)])
def test_writes_and_reads(dev, layout, dtype, q_heads, kv, dim, freqs):
    g = torch.Generator().manual_seed(dim)
    n, slots = 77, 100
    q, k, v = (torch.randn((n, h, dim), generator=g).to(dtype).to(dev) for h in (q_heads, kv, kv))
    inv = (1e4 ** (-torch.arange(freqs) / freqs)).to(dev)
    pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32).to(dev)
    at = torch.randperm(slots, generator=g)[:n].to(torch.int32).to(dev)
    w = (1 + 0.1 * torch.randn((2, dim), generator=g)).to(dev)
    how = dict(q_weight=w[0], k_weight=w[1])
    f = LAYOUTS[layout]
    dense = [torch.zeros((slots, kv, dim), dtype=dtype, device=dev) for _ in range(2)]
    want = gb.rotate_and_cache(q, k, v, pos, at, inv, *dense, **how)
    strided = [f(torch.zeros_like(x)) for x in dense]
    out = f(torch.zeros_like(q))
    assert gb.rotate_and_cache(f(q), f(k), f(v), pos, at, inv, *strided, q_out=out, **how) is out
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(strided, dense))
    rows = gb.int4_row_bytes(dim)
    c = torch.zeros((slots, kv, rows), dtype=torch.uint8, device=dev)
    assert torch.equal(gb.rotate_and_cache_int4(q, k, v, pos, at, inv, c, **how), want)
    big = torch.zeros((slots, 2 * kv + 1, rows + 16), dtype=torch.uint8, device=dev)
    d = big[:, 1::2, 16:]
    out = f(torch.zeros_like(q))
    gb.rotate_and_cache_int4(f(q), f(k), f(v), pos, at, inv, d, q_out=out, **how)
    assert torch.equal(out, want) and torch.equal(d, c)
    assert all(torch.equal(a, b) for a, b in zip(gb.read_cache_int4(c, at, dim, dtype), gb.read_cache_int4(d, at, dim, dtype)))


def test_rows_behind_the_whole_of_memory(dev):
    """Offsets beyond 32 bits: slots and rows far apart in one large tensor."""
    dim, kv, slots = 64, 2, 6
    far = 1 << 30                                              # elements between slots, 2 GB
    big = torch.zeros((slots * far,), dtype=BF, device=dev)
    kc, vc = (big.as_strided((slots, kv, dim), (far, dim, 1), o) for o in (0, far // 2))
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((slots, h, dim), generator=g).to(BF).to(dev) for h in (4, kv, kv))
    at = torch.arange(slots, dtype=torch.int32, device=dev)
    gb.rotate_and_cache(q, k, v, None, at, None, kc, vc)
    assert torch.equal(kc, k) and torch.equal(vc, v)
    cu = torch.tensor([0, slots], dtype=torch.int32, device=dev)
    assert torch.equal(gb.prompt_attention(q, kc, vc, cu), gb.prompt_attention(q, k, v, cu))
    bytes_ = big.view(torch.uint8)
    row = gb.int4_row_bytes(dim)
    dense = torch.zeros((slots, kv, row), dtype=torch.uint8, device=dev)
    gb.rotate_and_cache_int4(q, k, v, None, at, None, dense)
    step = 2 * far // row * row                                # a multiple of the rows
    c = bytes_.as_strided((slots, kv, row), (step, row, 1))
    c.zero_()                                                  # (a row's unused bytes stay as they are)
    gb.rotate_and_cache_int4(q, k, v, None, at, None, c)
    assert torch.equal(c, dense)
    assert all(torch.equal(a, b) for a, b in zip(gb.read_cache_int4(c, at, dim), gb.read_cache_int4(dense, at, dim)))
    pages, lens = at.view(1, -1), torch.tensor([slots], dtype=torch.int32, device=dev)
    assert torch.equal(gb.tree_attention_int4(q[:1], c, pages, lens), gb.tree_attention_int4(q[:1], dense, pages, lens))
    assert torch.equal(gb.selected_attention_int4(q[:1], c, pages), gb.selected_attention_int4(q[:1], dense, pages))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kv,dim", [(2, 128), (3, 48), (1, 256)])
def test_attention_over_parts_of_a_4_bit_cache(dev, dtype, kv, dim):
    """Every other slot, the last heads of more, heads outermost."""
    g = torch.Generator().manual_seed(dim)
    n, row = 500, gb.int4_row_bytes(dim)
    dense = torch.randint(0, 256, (n, kv, row), generator=g, dtype=torch.uint8).to(dev)
    dense[:, :, -2 * (8 if dim <= 128 else 16):] &= 0x3f         # (scales below 2)
    q = torch.randn((3, 4 * kv, dim), generator=g).to(dtype).to(dev)
    pages = torch.randperm(n, generator=g).to(torch.int32).to(dev).view(1, -1)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    want = gb.tree_attention_int4(q, dense, pages, lens, next_n=3, return_lse=True)
    listed = gb.selected_attention_int4(q, dense, pages[:, :200].repeat(3, 1), return_lse=True)
    big = torch.zeros((2 * n, kv + 2, row), dtype=torch.uint8, device=dev)
    for view in (big[::2, 2:], big[1::2, :kv], big.view(kv + 2, 2 * n, row).transpose(0, 1)[:n, 1:kv + 1]):
        view.copy_(dense)
        got = gb.tree_attention_int4(q, view, pages, lens, next_n=3, return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        got = gb.selected_attention_int4(q, view, pages[:, :200].repeat(3, 1), return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(got, listed))
