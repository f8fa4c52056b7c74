"""Decode-step operators at the ends of their ranges: positions close to 2^31,
temperatures close to zero and infinite."""
import math

import numpy as np
import pytest
import torch

import decode_reference as ref
import sparse_attention_top_gb300 as gb
from test_gpu_decode import BF, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gb.load_library()
    return torch.device("cuda:0")


def test_tree_attention_positions_close_to_31_bits(dev):
    """The last page of a table of 2^31 - 48 positions; its others do not exist.
    Outputs against the same page as a request of its own."""
    page, cols, next_n = 100, (2 ** 31 - 1) // 100, 3
    b = Batch([page], next_n, 4, 2, 64, page, BF, seed=12)
    k, v = b.caches(dev)
    table = torch.full((1, cols), -1, dtype=torch.int32, device=dev)
    table[0, -1] = b.table[0, 0]
    tree = np.array([1, 3, 5], dtype=np.int64)
    dtree = torch.from_numpy(tree).to(dev)
    lens = torch.tensor([cols * page], dtype=torch.int32, device=dev)
    out, lse = gb.tree_attention(b.q.to(dev), k, v, table, lens, page_size=page, next_n=next_n, tree_mask=dtree, return_lse=True)
    torch.cuda.synchronize(dev)
    q, kk, vv = b.wide()
    for r in range(next_n):
        seen = ref.visible(b.table.numpy(), page, k.shape[0], b.lens.numpy(), next_n, tree, r)
        o, l, eta, mag = ref.attend(q[r], kk, vv, seen, b.group, b.scale)
        tol = b.u * np.abs(o) + (b.u + 2 * eta[:, None]) * mag
        assert np.all(np.abs(out[r].cpu().double().numpy() - o) <= tol)
        assert np.all(np.abs(lse[r].cpu().double().numpy() - l) <= eta + 2.0 ** -21 * (1 + np.abs(l)))


@pytest.mark.parametrize("requests", [3, 700])
def test_verify_drafts_temperatures_at_the_ends(dev, requests):
    """A denormal temperature is greedy where the largest logit is alone; an
    infinite one makes the words that have a logit equal."""
    vocab, next_n = 5003, 3
    g = torch.Generator().manual_seed(requests)
    logits = torch.randn((requests * next_n, vocab), generator=g)
    logits[:, 7:2000] = -math.inf
    logits[torch.arange(requests * next_n), torch.randint(2000, vocab, (requests * next_n,), generator=g)] = 9.0
    tokens = torch.randint(0, vocab, (requests * next_n,), generator=g).to(torch.int32)
    tokens[1::next_n] = logits[0::next_n].argmax(1).to(torch.int32)
    u = torch.rand(requests * next_n, generator=g)
    noise = torch.empty((requests, vocab)).exponential_(generator=g).clamp_(min=1e-6)

    def run(x, t):
        got = gb.verify_drafts(x.to(dev), tokens.to(dev), u.to(dev), noise.to(dev), next_n=next_n,
                               temperature=torch.full((requests,), t, device=dev))
        return [a.cpu() for a in (got.accepted, got.path, got.next_token, got.accept_mask)]

    for a, b in zip(run(logits, 1e-42), run(logits, 0.0)):
        assert torch.equal(a, b)
    flat = torch.where(logits == -math.inf, logits, torch.zeros(()))
    for a, b in zip(run(logits, math.inf), run(flat, 1.0)):
        assert torch.equal(a, b)
