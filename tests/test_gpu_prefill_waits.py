"""Waits that run out in the attention over 4-bit caches and over prompts: calls
come back, say so in their workspace's status word, and leave nothing behind for
the next.  (In a process of its own, whose waits' limit is one cycle: a wait that
two tries do not end gives up.  A try sleeps for some microseconds, so the inputs
are such as make some warps wait for others for longer than they do as a rule.)"""
import os
import subprocess
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))      # as a child process too
import sparse_attention_top_gb300 as gb  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def _child():
    d = torch.device("cuda:0")
    g = torch.Generator(device=d).manual_seed(1)
    gave_up = {"4 bits": 0, "prompt": 0}
    calls = 0
    for dtype in (BF, HF):
        for dim, heads, kv in ((64, 8, 2), (128, 32, 4), (128, 64, 4), (256, 4, 1)):
            calls += 1
            # keys that grow along the context: every tile moves the references of its rows, which takes the longest
            n = 60000
            k = torch.randn((1, kv, dim), generator=g, device=d) * (1 + torch.arange(n, device=d) / 100.0).view(-1, 1, 1)
            cache = torch.zeros((n, kv, gb.int4_row_bytes(dim)), dtype=torch.uint8, device=d)
            q = torch.randn((1, heads, dim), generator=g, device=d).expand(8, -1, -1).to(dtype).contiguous()
            slots = torch.arange(n, dtype=torch.int32, device=d)
            gb.rotate_and_cache_int4(k.to(dtype), k.to(dtype), k.to(dtype), None, slots, None, cache)
            lens = torch.tensor([30000, 20000], dtype=torch.int32, device=d)
            ws = torch.zeros(gb.gbtopk_attention_workspace_bytes(8, heads, kv, dim), dtype=torch.uint8, device=d)
            gb.tree_attention_int4(q, cache, slots.view(2, 30000), lens, next_n=4, workspace=ws)
            torch.cuda.synchronize(d)
            status = gb.gbtopk_device_status(ws)
            assert status in (0, 2) and gb.gbtopk_device_status(ws) == 0
            gave_up["4 bits"] += status == 2
            # values that are no numbers: a unit's output adds each to the rows that see it, while the next unit's products wait
            x = torch.randn((3000, heads, dim), generator=g, device=d).to(dtype)
            y = torch.randn((3000, kv, dim), generator=g, device=d).to(dtype)
            z = torch.full((3000, kv, dim), float("inf"), dtype=dtype, device=d)
            cu = torch.tensor([0, 2500, 3000], dtype=torch.int32, device=d)
            ws = torch.zeros(gb.gbtopk_prompt_workspace_bytes(3000, 2, heads, kv, dim), dtype=torch.uint8, device=d)
            gb.prompt_attention(x, y, z, cu, workspace=ws)
            torch.cuda.synchronize(d)
            status = gb.gbtopk_device_status(ws)
            assert status in (0, 2) and gb.gbtopk_device_status(ws) == 0
            gave_up["prompt"] += status == 2
    print(gave_up, "of", calls)
    assert all(gave_up.values()), gave_up
    print("child: ok")


def test_some_calls_of_each_kind_give_up(dev):
    env = dict(os.environ, GBTOPK_WAIT_POLLS="1")
    r = subprocess.run([sys.executable, os.path.abspath(__file__), "child"], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "child: ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


if __name__ == "__main__" and len(sys.argv) > 1 and sys.argv[1] == "child":
    _child()
