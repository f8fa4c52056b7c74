"""The workspaces that the Python calls keep, on the GPU (see also
test_workspace_host)."""
import pytest
import torch

import sparse_attention_top_gb300 as gb
from test_gpu_decode_blocks import BF, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def test_a_captured_call_outlives_its_workspace(dev):
    """Replay after an eager call on the same stream needed a larger one: the
    outputs are the eager call's, and nothing that was allocated since is
    written to."""
    few, many = make(dev, [9000], 1, 8, 2, 128, 16, BF, 1), make(dev, [300] * 64, 4, 32, 2, 128, 16, BF, 2)

    def call(a, next_n):
        return gb.tree_attention(*a, page_size=16, next_n=next_n, return_lse=True)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        want = [x.clone() for x in call(few, 1)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = call(few, 1)
        before = gb.gbtopk_attention_workspace_bytes(1, 8, 2, 128)
        assert gb.gbtopk_attention_workspace_bytes(256, 32, 2, 128) > before
        call(many, 4)
        new = [torch.full((n,), 85, dtype=torch.uint8, device=dev) for n in (before, before // 2, before // 2, 1 << 22, 1 << 20)]
        for x in got:
            x.zero_()
        graph.replay()
    torch.cuda.synchronize(dev)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(bool((x == 85).all()) for x in new)
