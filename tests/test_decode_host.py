"""Refusals of the decode-step entry points: decided on the host, before
anything is enqueued (the addresses here are never dereferenced)."""
import pytest
import torch

import sparse_attention_top_gb300 as gb

A = 0x10000000


def call(name, order, defaults, **kw):
    a = dict(defaults)
    a.update(kw)
    assert set(a) == set(order)
    return getattr(gb.decode._lib(), name)(*[a[k] for k in order])


ATT = "q dtype rows q_row q_head q_heads kv_heads dim k k_slot k_head v v_slot v_head slots".split()
ATT_DEFAULTS = dict(q=A, dtype=1, rows=4, q_row=512, q_head=64, q_heads=8, kv_heads=2, dim=64, k=A, k_slot=128, k_head=64,
                    v=A, v_slot=128, v_head=64, slots=100)
TAIL = "scale out lse ws ws_bytes stream".split()
TAIL_DEFAULTS = dict(scale=1.0, out=A, lse=None, ws=A, ws_bytes=1 << 30, stream=None)
PAGES = "table cols pt_stride page lens next_n tree".split()
PAGES_DEFAULTS = dict(table=A, cols=7, pt_stride=7, page=16, lens=A, next_n=2, tree=None)


def tree(**kw):
    return call("gbtopk_tree_attention", ATT + PAGES + TAIL, {**ATT_DEFAULTS, **PAGES_DEFAULTS, **TAIL_DEFAULTS}, **kw)


def selected(**kw):
    return call("gbtopk_selected_attention", ATT + "idx top_k idx_stride".split() + TAIL,
                {**ATT_DEFAULTS, "idx": A, "top_k": 8, "idx_stride": 8, **TAIL_DEFAULTS}, **kw)


def weights(**kw):
    order = ATT[:11] + ["slots", "lse"] + PAGES + "accept scale weights w_heads width ws ws_bytes stream".split()
    d = {**ATT_DEFAULTS, **PAGES_DEFAULTS, "lse": A, "accept": None, "scale": 1.0, "weights": A, "w_heads": 1, "width": 64,
         "ws": A, "ws_bytes": 1 << 30, "stream": None}
    return call("gbtopk_cache_weights", order, {k: d[k] for k in order}, **kw)


def evict(**kw):
    order = ("weights requests w_heads width lens next_n accept budget recent k k_slot k_head v v_slot v_head slots kv_heads dim "
             "elem table cols pt_stride new_table new_cols new_stride page kept new_lens out_w stream").split()
    d = dict(weights=A, requests=2, w_heads=1, width=64, lens=A, next_n=1, accept=None, budget=32, recent=4, k=A, k_slot=128,
             k_head=64, v=A, v_slot=128, v_head=64, slots=100, kv_heads=2, dim=64, elem=2, table=A, cols=4, pt_stride=4,
             new_table=A, new_cols=2, new_stride=2, page=16, kept=A, new_lens=A, out_w=A + (1 << 20), stream=None)
    return call("gbtopk_cache_evict", order, d, **kw)


def verify(**kw):
    order = ("logits dtype rows vocab stride tokens uniforms noise next_n tree temperature draft accepted path next_token mask ws "
             "ws_bytes stream").split()
    d = dict(logits=A, dtype=0, rows=4, vocab=100, stride=100, tokens=A, uniforms=A, noise=A, next_n=2, tree=None,
             temperature=None, draft=None, accepted=A, path=A, next_token=A, mask=A, ws=A, ws_bytes=1 << 20, stream=None)
    return call("gbtopk_verify_drafts", order, d, **kw)


QUERY = [
    (dict(dtype=7), gb.EINVAL), (dict(dtype=0), gb.EUNSUPPORTED), (dict(rows=-2), gb.EINVAL),
    (dict(q_heads=0), gb.EINVAL), (dict(kv_heads=3), gb.EINVAL), (dict(kv_heads=0), gb.EINVAL),
    (dict(dim=0), gb.EINVAL), (dict(dim=60), gb.EUNSUPPORTED), (dict(dim=264), gb.EUNSUPPORTED),
    (dict(q=None), gb.EINVAL), (dict(k=None), gb.EINVAL), (dict(q=A + 8), gb.EALIGN), (dict(k=A + 2), gb.EALIGN),
    (dict(q_row=516), gb.EALIGN), (dict(k_slot=132), gb.EALIGN), (dict(k_head=-64), gb.EINVAL),
    (dict(slots=-1), gb.EINVAL), (dict(ws=None), gb.EWORKSPACE), (dict(ws=A + 16), gb.EWORKSPACE),
    (dict(ws_bytes=16), gb.EWORKSPACE),
]
PAGED = [
    (dict(next_n=0), gb.EINVAL), (dict(next_n=3), gb.EINVAL), (dict(rows=65 * 2, next_n=65), gb.EUNSUPPORTED),
    (dict(page=0), gb.EINVAL), (dict(cols=-1), gb.EINVAL), (dict(pt_stride=6), gb.EINVAL), (dict(table=None), gb.EINVAL),
    (dict(lens=None), gb.EINVAL),
]


@pytest.mark.parametrize("kw,status", QUERY + PAGED + [
    (dict(v=None), gb.EINVAL), (dict(v=A + 4), gb.EALIGN), (dict(v_slot=130), gb.EALIGN), (dict(out=None), gb.EINVAL),
    (dict(out=A + 2), gb.EALIGN), (dict(lse=A + 2), gb.EALIGN),
])
def test_tree_attention_refuses(kw, status):
    assert tree(**kw) == status


@pytest.mark.parametrize("kw,status", QUERY + [
    (dict(v=None), gb.EINVAL), (dict(idx=None), gb.EINVAL), (dict(top_k=-1), gb.EINVAL), (dict(idx_stride=7), gb.EINVAL),
    (dict(top_k=1 << 31, idx_stride=1 << 31), gb.EUNSUPPORTED), (dict(out=None), gb.EINVAL),
])
def test_selected_attention_refuses(kw, status):
    assert selected(**kw) == status


@pytest.mark.parametrize("kw,status", QUERY + PAGED + [
    (dict(w_heads=3), gb.EINVAL), (dict(width=-1), gb.EINVAL), (dict(lse=None), gb.EINVAL), (dict(weights=None), gb.EINVAL),
    (dict(weights=A + 4), gb.EALIGN), (dict(width=1 << 31), gb.EUNSUPPORTED),
])
def test_cache_weights_refuses(kw, status):
    assert weights(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(requests=-1), gb.EINVAL), (dict(w_heads=3), gb.EINVAL), (dict(budget=0), gb.EINVAL), (dict(recent=-1), gb.EINVAL),
    (dict(budget=33), gb.EINVAL), (dict(page=0), gb.EINVAL), (dict(next_n=0), gb.EINVAL), (dict(next_n=65), gb.EUNSUPPORTED),
    (dict(elem=1), gb.EUNSUPPORTED), (dict(dim=60), gb.EALIGN), (dict(k=A + 8), gb.EALIGN), (dict(v_slot=130), gb.EALIGN),
    (dict(weights=None), gb.EINVAL), (dict(lens=None), gb.EINVAL), (dict(new_table=None), gb.EINVAL),
    (dict(table=None), gb.EINVAL), (dict(kept=None), gb.EINVAL), (dict(new_lens=None), gb.EINVAL), (dict(out_w=None), gb.EINVAL),
    (dict(out_w=A + 64), gb.EOVERLAP), (dict(pt_stride=3), gb.EINVAL), (dict(new_stride=1), gb.EINVAL), (dict(slots=-1), gb.EINVAL),
])
def test_cache_evict_refuses(kw, status):
    assert evict(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=9), gb.EINVAL), (dict(rows=-1), gb.EINVAL), (dict(vocab=0), gb.EINVAL), (dict(next_n=3), gb.EINVAL),
    (dict(rows=130, next_n=65), gb.EUNSUPPORTED), (dict(stride=99), gb.EINVAL), (dict(draft=A, tree=A), gb.EINVAL),
    (dict(logits=None), gb.EINVAL), (dict(noise=None), gb.EINVAL), (dict(tokens=None), gb.EINVAL),
    (dict(uniforms=None), gb.EINVAL), (dict(mask=None), gb.EINVAL), (dict(logits=A + 2), gb.EALIGN),
    (dict(mask=A + 4), gb.EALIGN), (dict(ws=None), gb.EWORKSPACE), (dict(ws_bytes=10), gb.EWORKSPACE),
])
def test_verify_drafts_refuses(kw, status):
    assert verify(**kw) == status


def test_no_rows_is_a_noop():
    assert tree(rows=0, q=None, k=None, v=None, out=None, ws=None, table=None, lens=None) == gb.OK
    assert selected(rows=0, q=None, k=None, v=None, out=None, ws=None, idx=None) == gb.OK
    assert weights(rows=0, q=None, k=None, lse=None, weights=None, ws=None, table=None, lens=None) == gb.OK
    assert evict(requests=0, weights=None, k=None, v=None) == gb.OK
    assert verify(rows=0, logits=None, ws=None) == gb.OK


def test_workspace_sizes():
    assert gb.gbtopk_attention_workspace_bytes(4, 8, 2, 64) >= 256
    assert gb.gbtopk_attention_workspace_bytes(4, 8, 3, 64) == 0
    assert gb.gbtopk_verify_workspace_bytes(64, 1000, 4) >= 256
    assert gb.gbtopk_verify_workspace_bytes(64, 1000, 5) == 0


def test_python_checks():
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):         # there is no CPU path
        gb.tree_attention(q, q, q, torch.zeros((2, 1), dtype=torch.int32), torch.ones(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        gb.verify_drafts(torch.zeros((2, 9)), torch.zeros(2, dtype=torch.int32), torch.zeros(2), torch.zeros((2, 9)))


@pytest.mark.parametrize("new_lens,status", [(A, gb.EOVERLAP), (A + 4, gb.EOVERLAP), (A - 4, gb.EOVERLAP)])
def test_cache_evict_refuses_lengths_in_place(new_lens, status):
    """A request's heads read its length at different times."""
    assert evict(lens=A, new_lens=new_lens) == status


@pytest.mark.parametrize("call,kw", [
    (tree, dict(table=A + 2)), (tree, dict(lens=A + 1)), (tree, dict(tree=A + 4)),
    (selected, dict(idx=A + 2)),
    (weights, dict(table=A + 2)), (weights, dict(lens=A + 2)), (weights, dict(tree=A + 4)), (weights, dict(accept=A + 4)),
    (weights, dict(lse=A + 2)),
    (evict, dict(lens=A + 18)), (evict, dict(accept=A + 4)), (evict, dict(table=A + 2)), (evict, dict(new_table=A + 2)),
    (evict, dict(new_lens=A + 18)),
    (verify, dict(tokens=A + 2)), (verify, dict(uniforms=A + 2)), (verify, dict(tree=A + 4)), (verify, dict(temperature=A + 2)),
    (verify, dict(draft=A + 2)), (verify, dict(path=A + 2)),
])
def test_arrays_off_their_types_boundary_are_refused(call, kw):
    assert call(**kw) == gb.EALIGN
