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


# ------------------------------------------------------ two host threads

BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


class Library:
    """Stands in for the C calls: `hold(name, address)` runs inside each."""

    def __init__(self, hold):
        self.hold = hold

    def __getattr__(self, name):
        def call(*args):
            self.hold(name, args[-3])     # workspace, its bytes, stream
            return 0
        return call


def attention(rows):
    q, cache = fake(rows, 4, 64, dtype=BF), fake(32, 2, 64, dtype=BF)
    return q, cache, fake(rows, 1, dtype=I32), fake(rows, dtype=I32), fake(rows, 4)


def tree(rows):
    q, cache, table, lens, lse = attention(rows)
    gb.tree_attention(q, cache, cache, table, lens, page_size=32, out=fake(rows, 4, 64, dtype=BF), lse=lse)


def selected(rows):
    q, cache, table, _, lse = attention(rows)
    gb.selected_attention(q, cache, cache, table, out=fake(rows, 4, 64, dtype=BF), lse=lse)


def weights(rows):
    q, cache, table, lens, lse = attention(rows)
    gb.accumulate_cache_weights(q, cache, lse, table, lens, fake(rows, 2, 32), page_size=32)


def verify(rows):
    gb.verify_drafts(fake(rows, 9), fake(rows, dtype=I32), fake(rows), fake(rows, 9))


def top_k(rows):
    gb.top_k_varlen(fake(rows, 40), fake(rows, dtype=I32), 4, out_indices=fake(rows, 4, dtype=I32))


def pages(rows):
    gb.top_k_page_table_transform(fake(rows, 40), fake(rows, dtype=I32), fake(rows, 40, dtype=I32), 4,
                                  out=fake(rows, 4, dtype=I32))


CALLS = [tree, selected, weights, verify, top_k, pages]


@pytest.fixture
def library(made, monkeypatch):
    """install(hold): the C calls are hold's, the workspaces grow with the rows."""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    for at, name in ((gb.decode, "_attention_bytes"), (gb.decode, "_verify_bytes"), (gb, "gbtopk_workspace_bytes")):
        monkeypatch.setattr(at, name, lambda rows, *a: 1000 * rows)

    def install(hold):
        lib = Library(hold)
        monkeypatch.setattr(gb.decode, "_calls", lib)
        monkeypatch.setattr(gb, "load_library", lambda: lib)
    return install


def run(*jobs):
    failed = []

    def go(job):
        try:
            job()
        except BaseException as e:      # noqa: B902
            failed.append(e)
    threads = [threading.Thread(target=go, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed, failed


@pytest.mark.parametrize("call", CALLS)
def test_a_workspace_is_one_calls_until_it_is_enqueued(library, made, call):
    """Two threads on one stream, one of them with growing calls: the tensor
    stays and no other call comes between, while the first is in the library."""
    inside, gate, seen = [], threading.Event(), []

    def hold(name, address):
        inside.append(address)
        seen.append((len(inside), made[address]() is not None))
        gate.wait(0.1 if len(seen) < 3 else 0.001)     # long enough for the other thread to come in
        seen.append((len(inside), made[address]() is not None))
        inside.remove(address)
    library(hold)
    run(lambda: [call(1) for _ in range(4)], lambda: [call(n) for n in (2, 20, 200)])
    assert len(seen) == 14 and all(s == (1, True) for s in seen), seen


def test_calls_on_two_streams_do_not_wait_for_one_another(library, made, monkeypatch):
    stream = threading.local()
    monkeypatch.setattr(gb, "_stream_handle", lambda device: stream.handle)
    both = threading.Barrier(2)
    library(lambda name, address: both.wait(30))

    def job(handle):
        stream.handle = handle
        tree(1)
    run(lambda: job(3), lambda: job(4))


def test_a_call_that_fails_gives_its_workspace_back(library, made, monkeypatch):
    library(lambda name, address: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError):
        tree(1)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)

    def fails(name, address):
        raise OSError
    library(fails)
    with pytest.raises(OSError):
        tree(1)
    library(lambda name, address: None)
    run(lambda: tree(1))


# ------------------------------------------------------ another device's tensors

class Other(Fake):
    device = property(lambda self: torch.device("cuda:1"))


def evict(rows):
    cache, table = fake(64, 2, 64, dtype=BF), fake(rows, 1, dtype=I32)
    gb.evict_cache(fake(rows, 2, 32), cache, cache, table, fake(rows, dtype=I32), table, 8, page_size=32,
                   out_weights=fake(rows, 2, 32))


def direct(rows):
    gb.gbtopk_varlen(fake(rows, 40), fake(rows, dtype=I32), 4, None, 1, 1, fake(rows, 4, dtype=I32), None, 0,
                     fake(1000, dtype=torch.uint8))


def direct_on_a_stream(rows):
    gb.gbtopk_varlen(fake(rows, 40), fake(rows, dtype=I32), 4, None, 1, 1, fake(rows, 4, dtype=I32), None, 0,
                     fake(1000, dtype=torch.uint8), stream=5)


@pytest.mark.parametrize("call", CALLS + [evict, direct, direct_on_a_stream])
def test_tensors_of_a_device_that_is_not_current_are_refused(made, monkeypatch, call):
    """The library launches on the current device."""
    monkeypatch.undo()
    calls, empty, zeros = [], torch.empty, torch.zeros
    lib = Library(lambda name, address: calls.append(name))
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    monkeypatch.setattr(gb, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(gb, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(gb, "_WS", {})
    for at, name in ((gb.decode, "_attention_bytes"), (gb.decode, "_verify_bytes"), (gb, "gbtopk_workspace_bytes")):
        monkeypatch.setattr(at, name, lambda rows, *a: 1000 * rows)
    monkeypatch.setattr(gb.decode, "_calls", lib)
    monkeypatch.setattr(gb, "load_library", lambda: lib)
    call(1)                                     # on the current device it goes through
    assert len(calls) == 1
    monkeypatch.setattr("test_workspace_host.Fake", Other)
    with pytest.raises(ValueError, match="current device"):
        call(1)
    assert len(calls) == 1


# ------------------------------------------------------ a caller's workspace

def given(call, workspace, monkeypatch):
    """The call with that workspace: its kernels' address, or None if refused."""
    seen = []
    lib = Library(lambda name, address: seen.append(address))
    monkeypatch.setattr(gb.decode, "_calls", lib)
    monkeypatch.setattr(gb, "load_library", lambda: lib)
    for at, name in ((gb, "top_k_varlen"), (gb, "top_k_page_table_transform"), (gb, "tree_attention"),
                     (gb, "selected_attention"), (gb, "accumulate_cache_weights"), (gb, "verify_drafts")):
        real = getattr(at, name)
        monkeypatch.setattr(at, name, lambda *a, real=real, **k: real(*a, workspace=workspace, **k))
    try:
        call(1)
    except ValueError:
        return None
    return seen[0]


@pytest.mark.parametrize("call", CALLS)
def test_a_callers_workspace_has_to_own_its_bytes(library, monkeypatch, call):
    monkeypatch.setattr(gb, "_current_device", lambda: 0)
    good = fake(4096, dtype=torch.uint8)
    for ok, ws in ((True, good), (False, good[:1].expand(4096)), (False, good[::2]), (False, torch.zeros(4096, dtype=torch.uint8)),
                   (False, torch.Tensor._make_subclass(Other, torch.empty(4096, dtype=torch.uint8)))):
        with monkeypatch.context() as m:
            assert given(call, ws, m) == (ws.data_ptr() if ok else None)
    assert not gb._WS


# ------------------------------------------------------ numbers beyond the C types

def evicted(page_size=32, next_n=1, budget=8, recent=0, cols=1):
    cache, table = fake(64, 2, 64, dtype=BF), fake(1, cols, dtype=I32)
    gb.evict_cache(fake(1, 2, 32), cache, cache, table, fake(1, dtype=I32), table, budget, recent=recent, page_size=page_size,
                   next_n=next_n, out_weights=fake(1, 2, 32))


def paged(page_size):
    q, cache, table, lens, lse = attention(1)
    gb.tree_attention(q, cache, cache, table, lens, page_size=page_size, out=fake(1, 4, 64, dtype=BF), lse=lse)


def weighed(page_size):
    q, cache, table, lens, lse = attention(1)
    gb.accumulate_cache_weights(q, cache, lse, table, lens, fake(1, 2, 32), page_size=page_size)


@pytest.mark.parametrize("call,good,bad", [
    (paged, 32, 2 ** 32 + 32), (paged, 2 ** 30, 2 ** 30 + 1), (paged, 1, 0), (weighed, 32, 2 ** 32 + 32), (weighed, 1, -1),
    (lambda n: evicted(page_size=n), 32, 2 ** 32 + 32), (lambda n: evicted(next_n=n), 64, 2 ** 32 + 1),
    (lambda n: evicted(budget=n, page_size=2 ** 30, cols=5), 100, 2 ** 32 + 8),
    (lambda n: evicted(recent=n), 2 ** 31 - 1, 2 ** 32),
])
def test_numbers_that_the_library_cannot_hold_are_refused(library, monkeypatch, call, good, bad):
    monkeypatch.setattr(gb, "_current_device", lambda: 0)
    seen = []
    library(lambda name, address: seen.append(name))
    call(good)
    assert len(seen) == 1
    with pytest.raises(ValueError):
        call(bad)
    assert len(seen) == 1
