"""The workspaces that the Python calls keep, on the GPU (see also
test_workspace_host)."""
import threading

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


def test_two_host_threads_on_one_stream(dev):
    """Calls whose parts are joined by a second kernel, from two threads, one
    with batches that grow: every output is the same call's alone, to the bit."""
    batches = [[make(dev, [9000 + 50 * i], 2, 8, 1, 128, 16, BF, i) for i in range(3)],
               [make(dev, [5000] * (i + 1), 4, 16, 2, 128, 16, BF, 10 + i) for i in range(6)]]
    tokens = [2, 4]

    def call(which, a):
        return gb.tree_attention(*a, page_size=16, next_n=tokens[which], return_lse=True)
    want = [[[x.clone() for x in call(w, a)] for a in b] for w, b in enumerate(batches)]
    torch.cuda.synchronize(dev)
    gb._WS.pop((dev.index, gb._stream_handle(dev)))     # start from a small one again
    wrong, failed = [], []

    def job(which):
        try:
            torch.cuda.set_device(dev)
            for turn in range(40):
                got = [call(which, a) for a in batches[which]]
                torch.cuda.synchronize(dev)
                wrong.extend((which, turn, i) for i, (g, w) in enumerate(zip(got, want[which]))
                             if not all(torch.equal(x, y) for x, y in zip(g, w)))
        except BaseException as e:      # noqa: B902
            failed.append(e)
    threads = [threading.Thread(target=job, args=(w,)) for w in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed and not wrong, (failed, wrong[:5])
