"""What the top-k calls write is there for the decode-step calls behind them
on the stream, whichever kernels of a launch plan had nothing to do."""
import pytest
import torch

import sparse_attention_top_gb300 as gb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("rows,width,fused", [(64, 163840, 1), (32, 40000, 1), (600, 70000, 0)])
def test_attention_behind_a_selection_of_short_rows(dev, rows, width, fused):
    """Early in every request: a split launch plan none of whose rows is
    longer than top_k, eagerly and replayed, over other slots each time."""
    top_k = 2048
    assert gb.gbtopk_plan_query(rows, width, top_k, torch.float32)["fused"] == fused
    g = torch.Generator(device=dev).manual_seed(rows)
    scores = torch.randn((rows, width), generator=g, device=dev)
    slots = 4 * top_k
    k = torch.randn((slots, 1, 64), generator=g, device=dev).to(torch.bfloat16)
    v = torch.randn(k.shape, generator=g, device=dev).to(torch.bfloat16)
    q = torch.randn((rows, 4, 64), generator=g, device=dev).to(torch.bfloat16)
    table = torch.empty((rows, width), dtype=torch.int32, device=dev)
    lens = torch.empty(rows, dtype=torch.int32, device=dev)
    idx, out = torch.empty((rows, top_k), dtype=torch.int32, device=dev), torch.empty_like(q)

    def step():
        gb.top_k_page_table_transform(scores, lens, table, top_k, out=idx, deterministic=True)
        gb.selected_attention(q, k, v, idx, out=out)

    def check(turn):
        idx.fill_(turn % slots)                     # what a reader that comes too early finds
        table.random_(0, slots, generator=g)
        lens.copy_(torch.randint(0, top_k + 1, (rows,), generator=g, device=dev))
        yield
        torch.cuda.synchronize(dev)
        assert torch.equal((idx >= 0).sum(1).to(torch.int32), lens)
        assert torch.equal(out, gb.selected_attention(q, k, v, idx)), turn
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        for turn in range(20):
            for _ in check(turn):
                step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for turn in range(20, 60):
            for _ in check(turn):
                graph.replay()
