"""The prompt's operators with one another and with the decode step's: a run of
them together, caches moved by the eviction, calls on other streams and from
two host threads, captured calls, and waits that run out."""
import os
import subprocess
import sys
import threading

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import sparse_attention_top_gb300 as gb  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("prompt,four_bit", [(60, False), (0, True), (100, True)])
def test_example_runs(dev, prompt, four_bit):
    import decode_step
    lines = []
    said = decode_step.run(steps=12, batch=3, say=lines.append, prompt=prompt, four_bit=four_bit)
    assert len(lines) == 12 and all(0 <= t < decode_step.VOCAB for words in said for t in words)
    assert said == decode_step.run(steps=12, batch=3, say=lambda s: None, prompt=prompt, four_bit=four_bit)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_prompt_then_tokens_agree_with_one_longer_prompt(dev, dtype):
    """Keys and values rotated, cached, read back; the prompt's last tokens again
    as a chunk over the context, and as drafts over the paged cache: all of
    them are the same attention (each within its own rounding of the others)."""
    g = torch.Generator(device=dev).manual_seed(3)
    n, drafts, heads, kv, dim, page = 300, 5, 8, 2, 128, 16
    x = torch.randn((n, heads + 2 * kv, dim), generator=g, device=dev).to(dtype)
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    table = torch.randperm(30, generator=g, device=dev)[:19].to(torch.int32).view(1, 19)
    pos = torch.arange(n, device=dev, dtype=torch.int32)
    slots = (table[0, (pos // page).long()] * page + pos % page).to(torch.int32)
    freqs = 1e4 ** (-torch.arange(64, device=dev) / 64)
    w = torch.ones(dim, device=dev)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    for four_bit in (False, True):
        if four_bit:
            cache = torch.zeros((480, kv, gb.int4_row_bytes(dim)), dtype=torch.uint8, device=dev)
            turned = gb.rotate_and_cache_int4(q, k, v, pos, slots, freqs, cache, q_weight=w, k_weight=w)
            ck, cv = gb.read_cache_int4(cache, slots, dim, dtype)
        else:
            kc, vc = torch.zeros((2, 480, kv, dim), dtype=dtype, device=dev)
            turned = gb.rotate_and_cache(q, k, v, pos, slots, freqs, kc, vc, q_weight=w, k_weight=w)
            ck, cv = kc[slots.long()], vc[slots.long()]
        whole = gb.prompt_attention(turned, ck, cv, cu, return_lse=True)
        tail = turned[n - drafts:].contiguous()
        chunk = gb.prompt_attention(tail, ck, cv, torch.tensor([0, drafts], dtype=torch.int32, device=dev), cu_seqlens_k=cu, return_lse=True)
        args = (table, lens)
        if four_bit:
            tree = gb.tree_attention_int4(tail, cache, *args, page_size=page, next_n=drafts, return_lse=True)
            one = gb.selected_attention_int4(tail[-1:], cache, slots.view(1, -1), return_lse=True)
        else:
            tree = gb.tree_attention(tail, kc, vc, *args, page_size=page, next_n=drafts, return_lse=True)
            one = gb.selected_attention(tail[-1:], kc, vc, slots.view(1, -1), return_lse=True)
        # every call is off by its rounding of out and of each probability: u |out| + u sum p |v|, |v| below 6
        u = 2.0 ** -8 if dtype is BF else 2.0 ** -11
        for a, b in ((whole[0][-drafts:], chunk[0]), (whole[0][-drafts:], tree[0]), (whole[0][-1:], one[0])):
            assert float((a.float() - b.float()).abs().max()) <= 2 * u * 12
        for a, b in ((whole[1][-drafts:], chunk[1]), (whole[1][-drafts:], tree[1]), (whole[1][-1:], one[1])):
            assert float((a - b).abs().max()) < 1e-4


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("heads", [1, 3])
def test_eviction_moves_rows_whole(dev, dim, heads):
    g = torch.Generator(device=dev).manual_seed(dim)
    n = gb.int4_row_bytes(dim)
    cache = torch.randint(0, 256, (400, 3, n), generator=g, device=dev, dtype=torch.uint8)
    before = cache.clone()
    table = torch.arange(0, 12, device=dev, dtype=torch.int32).view(1, 12)
    new = torch.arange(20, 24, device=dev, dtype=torch.int32).view(1, 4)
    lens = torch.tensor([180], dtype=torch.int32, device=dev)
    weights = torch.rand((1, heads, 192), generator=g, device=dev)
    got = gb.evict_cache(weights, *gb.int4_parts(cache), table, lens, new, 60, recent=10, page_size=16)
    for h in range(3):
        kept = got.kept[0, h if heads > 1 else 0].long()
        assert torch.equal(cache[320:320 + 60, h], before[kept, h])
    assert torch.equal(cache[:320], before[:320]) and torch.equal(cache[380:], before[380:])
    with pytest.raises(ValueError):
        gb.int4_parts(cache[..., :n - 8])


def calls(dev, seed):
    """One of each operator, its inputs made before it; a list of outputs."""
    g = torch.Generator(device=dev).manual_seed(seed)
    n, heads, kv, dim = 200 + seed, 8, 2, 64
    x = torch.randn((n, heads + 2 * kv, dim), generator=g, device=dev).to(BF)
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    slots = torch.randperm(512, generator=g, device=dev)[:n].to(torch.int32)
    pos = torch.arange(n, device=dev, dtype=torch.int32)
    freqs = 1e4 ** (-torch.arange(32, device=dev) / 32)
    cache = torch.zeros((512, kv, gb.int4_row_bytes(dim)), dtype=torch.uint8, device=dev)
    cu = torch.tensor([0, 77, n], dtype=torch.int32, device=dev)
    table = slots.view(1, -1)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)

    def run():
        turned = gb.rotate_and_cache_int4(q, k, v, pos, slots, freqs, cache)
        ck, cv = gb.read_cache_int4(cache, slots, dim)
        a = gb.prompt_attention(turned, ck, cv, cu, return_lse=True)
        b = gb.tree_attention_int4(turned[:4].contiguous(), cache, table, lens, next_n=4, return_lse=True)
        c = gb.selected_attention_int4(turned[:4].contiguous(), cache, table[:, :100].repeat(4, 1))
        return [turned, ck, cv, *a, *b, c]
    return run


def test_streams_threads_and_graphs(dev):
    """The same results on side streams, from two host threads at once, and from
    two captured graphs that are replayed in turn."""
    runs = [calls(dev, s) for s in (1, 40)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize(dev)
    problems = []

    def work(i):
        try:
            with torch.cuda.device(dev), torch.cuda.stream(torch.cuda.Stream(dev)):
                for _ in range(30):
                    got = runs[i]()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    problems.append(i)
        except Exception as e:      # noqa: BLE001
            problems.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not problems, problems
    stream, graphs = torch.cuda.Stream(dev), []
    with torch.cuda.stream(stream):
        for r in runs:
            r()
        stream.synchronize()
        for r in runs:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                graphs.append((graph, r()))
            graphs[-1] = (graph, graphs[-1][1])
        for i in (0, 1, 1, 0):
            graphs[i][0].replay()
            stream.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(graphs[i][1], want[i]))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim,q_heads,next_n", [(16, 4, 2), (48, 8, 2), (64, 8, 1), (64, 8, 4), (64, 16, 4), (96, 4, 1)])
def test_calls_end_when_their_work_has(dev, dtype, dim, q_heads, next_n):
    """Many tiles a block, more than its ring has stages, of several lengths: no
    block waits for a copy that ended long ago (a wait's limit is about a second)."""
    g = torch.Generator(device=dev).manual_seed(dim)
    cache = torch.randint(0, 256, (60000, 1, gb.int4_row_bytes(dim)), generator=g, device=dev, dtype=torch.uint8)
    q = torch.randn((8 * next_n, q_heads, dim), generator=g, device=dev).to(dtype)
    table = torch.arange(60000, device=dev, dtype=torch.int32).expand(8, -1).contiguous()
    gb.tree_attention_int4(q[:next_n], cache, table[:1], torch.ones(1, dtype=torch.int32, device=dev), next_n=next_n)
    torch.cuda.synchronize(dev)
    for n in (12000, 27000, 41000, 60000):
        lens = torch.full((8,), n, dtype=torch.int32, device=dev)
        ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ends[0].record()
        gb.tree_attention_int4(q, cache, table, lens, next_n=next_n)
        ends[1].record()
        torch.cuda.synchronize(dev)
        assert ends[0].elapsed_time(ends[1]) < 200


def _child():
    """A process whose waits run out almost at once: every call comes back, and
    one that gave up says so in its workspace's status word."""
    d = torch.device("cuda:0")
    g = torch.Generator(device=d).manual_seed(1)
    for dim, heads, kv in ((64, 8, 2), (128, 32, 4), (256, 4, 1)):
        cache = torch.randint(0, 256, (60000, kv, gb.int4_row_bytes(dim)), generator=g, device=d, dtype=torch.uint8)
        table = torch.arange(60000, device=d, dtype=torch.int32).view(2, 30000)
        lens = torch.tensor([30000, 20000], dtype=torch.int32, device=d)
        q = torch.randn((8, heads, dim), generator=g, device=d).to(BF)
        ws = torch.zeros(gb.gbtopk_attention_workspace_bytes(8, heads, kv, dim), dtype=torch.uint8, device=d)
        gb.tree_attention_int4(q, cache, table, lens, next_n=4, workspace=ws)
        torch.cuda.synchronize(d)
        assert gb.gbtopk_device_status(ws) in (0, 2) and gb.gbtopk_device_status(ws) == 0
        x = torch.randn((3000, heads, dim), generator=g, device=d).to(BF)
        y = torch.randn((3000, kv, dim), generator=g, device=d).to(BF)
        cu = torch.tensor([0, 2500, 3000], dtype=torch.int32, device=d)
        ws = torch.zeros(gb.gbtopk_prompt_workspace_bytes(3000, 2, heads, kv, dim), dtype=torch.uint8, device=d)
        gb.prompt_attention(x, y, y, cu, workspace=ws)
        torch.cuda.synchronize(d)
        assert gb.gbtopk_device_status(ws) in (0, 2) and gb.gbtopk_device_status(ws) == 0
    print("child: ok")


def test_waits_that_run_out_end_the_call(dev):
    env = dict(os.environ, GBTOPK_WAIT_POLLS="1")
    r = subprocess.run([sys.executable, os.path.abspath(__file__), "child"], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "child: ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


if __name__ == "__main__" and len(sys.argv) > 1 and sys.argv[1] == "child":
    _child()
