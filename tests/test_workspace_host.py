"""The workspaces that the Python calls keep, one a stream: who holds them and
how long.  On the host alone: tensors that say they are on a GPU, and a
library whose calls only note what they were given."""
import threading
import weakref

import pytest
import torch

import sparse_attention_top_gb300 as gb

GPU = torch.device("cuda:0")


class Fake(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    device = property(lambda self: GPU)
    is_cuda = property(lambda self: True)


def fake(*shape, dtype=torch.float32):
    return torch.Tensor._make_subclass(Fake, torch.empty(shape, dtype=dtype))


@pytest.fixture
def made(monkeypatch):
    """Weak references to the workspaces made, by address."""
    refs, real = {}, torch.zeros

    def zeros(*size, dtype=None, device=None):
        t = real(*size, dtype=dtype)
        refs[t.data_ptr()] = weakref.ref(t)
        return t
    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(gb, "_stream_handle", lambda device: 7)
    monkeypatch.setattr(gb, "_WS", {})
    return refs


def test_an_outgrown_workspace_stays(made):
    """A captured graph may still write to it."""
    sizes = [1000, 999, 1001, 1500, 2000, 100000]
    at = [gb._workspace(GPU, n).data_ptr() for n in sizes]
    assert at[0] == at[1] and at[2] == at[3] == at[4] != at[0]
    assert len(made) == 3 and all(r() is not None for r in made.values())
    held = [made[a]().numel() for a in dict.fromkeys(at)]
    assert held[0] == 1000 and held[1] >= 2 * held[0] and held[2] >= 2 * held[1]


def test_a_capture_needs_a_workspace_that_is_there(made, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError):
        gb._workspace(GPU, 1000)
