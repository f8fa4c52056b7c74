"""Refusals of the prompt's entry points: decided on the host, before anything
is enqueued (the addresses here are never dereferenced)."""
import math

import pytest

import sparse_attention_top_gb300 as gb

A = 0x10000000


def call(name, order, defaults, **kw):
    a = dict(defaults)
    a.update(kw)
    assert set(a) == set(order)
    return getattr(gb.prefill._lib(), name)(*[a[k] for k in order])


TOKENS = ("q dtype rows q_row q_head k k_row k_head v v_row v_head q_heads kv_heads dim positions freq freqs pairs wq wk wtype eps "
          "q_out qo_row qo_head slots").split()
TOKENS_DEFAULTS = dict(q=A, dtype=1, rows=4, q_row=768, q_head=64, k=A, k_row=768, k_head=64, v=A, v_row=768, v_head=64, q_heads=8,
                       kv_heads=2, dim=64, positions=A, freq=A, freqs=32, pairs=0, wq=A, wk=A, wtype=1, eps=1e-6, q_out=A,
                       qo_row=512, qo_head=64, slots=A)


def rotate(**kw):
    return call("gbtopk_rotate_and_cache", TOKENS + "kc k_slot kc_head vc v_slot vc_head n stream".split(),
                {**TOKENS_DEFAULTS, "kc": A, "k_slot": 128, "kc_head": 64, "vc": A, "v_slot": 128, "vc_head": 64, "n": 50,
                 "stream": None}, **kw)


def rotate4(**kw):
    return call("gbtopk_rotate_and_cache_int4", TOKENS + "cache slot head n ks vs stream".split(),
                {**TOKENS_DEFAULTS, "cache": A, "slot": 160, "head": 80, "n": 50, "ks": 1.0, "vs": 1.0, "stream": None}, **kw)


def read(**kw):
    return call("gbtopk_cache_read_int4", "cache slot head n kv_heads dim slots listed ks vs dtype k v stream".split(),
                dict(cache=A, slot=160, head=80, n=50, kv_heads=2, dim=64, slots=A, listed=7, ks=1.0, vs=1.0, dtype=1, k=A, v=A,
                     stream=None), **kw)


SHARED = [
    (dict(dtype=7), gb.EINVAL), (dict(dtype=0), gb.EUNSUPPORTED), (dict(rows=-1), gb.EINVAL), (dict(q_heads=0), gb.EINVAL),
    (dict(kv_heads=3), gb.EINVAL), (dict(dim=0), gb.EINVAL), (dict(dim=60), gb.EUNSUPPORTED), (dict(dim=272), gb.EUNSUPPORTED),
    (dict(q=None), gb.EINVAL), (dict(k=None), gb.EINVAL), (dict(v=None), gb.EINVAL), (dict(q_out=None), gb.EINVAL),
    (dict(q=A + 8), gb.EALIGN), (dict(v_row=770), gb.EALIGN), (dict(qo_head=4), gb.EALIGN), (dict(k_head=-8), gb.EINVAL),
    (dict(positions=None), gb.EINVAL), (dict(freq=None), gb.EINVAL), (dict(freqs=40), gb.EINVAL), (dict(freqs=-8), gb.EINVAL),
    (dict(freqs=12), gb.EUNSUPPORTED), (dict(wtype=2), gb.EUNSUPPORTED), (dict(wq=A + 4), gb.EALIGN), (dict(eps=-1.0), gb.EINVAL),
    (dict(eps=math.nan), gb.EINVAL), (dict(slots=None), gb.EINVAL), (dict(slots=A + 2), gb.EALIGN), (dict(n=-1), gb.EINVAL),
    (dict(n=1 << 31), gb.EUNSUPPORTED), (dict(rows=1 << 31), gb.EUNSUPPORTED), (dict(positions=A + 1), gb.EALIGN),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(kc=None), gb.EINVAL), (dict(vc=A + 2), gb.EALIGN), (dict(k_slot=132), gb.EALIGN), (dict(vc_head=-64), gb.EINVAL)])
def test_rotate_and_cache_refuses(kw, status):
    assert rotate(**kw) == status


UNITS = [(dict(ks=0.0), gb.EINVAL), (dict(ks=3.0), gb.EINVAL), (dict(vs=-2.0), gb.EINVAL), (dict(vs=math.inf), gb.EINVAL),
         (dict(vs=math.nan), gb.EINVAL), (dict(ks=2.0 ** 61), gb.EINVAL), (dict(ks=2.0 ** -61), gb.EINVAL)]


@pytest.mark.parametrize("kw,status", SHARED + UNITS + [
    (dict(cache=None), gb.EINVAL), (dict(cache=A + 8), gb.EALIGN), (dict(slot=168), gb.EALIGN), (dict(head=-80), gb.EINVAL),
    (dict(dim=72, freqs=0), gb.EUNSUPPORTED)])
def test_rotate_and_cache_int4_refuses(kw, status):
    assert rotate4(**kw) == status


@pytest.mark.parametrize("kw,status", UNITS + [
    (dict(dtype=0), gb.EUNSUPPORTED), (dict(dtype=5), gb.EINVAL), (dict(dim=72), gb.EUNSUPPORTED), (dict(kv_heads=0), gb.EINVAL),
    (dict(cache=None), gb.EINVAL), (dict(cache=A + 4), gb.EALIGN), (dict(slot=72), gb.EALIGN), (dict(listed=-1), gb.EINVAL),
    (dict(listed=1 << 31), gb.EUNSUPPORTED), (dict(slots=None), gb.EINVAL), (dict(k=None), gb.EINVAL), (dict(v=None), gb.EINVAL),
    (dict(slots=A + 1), gb.EALIGN), (dict(v=A + 8), gb.EALIGN), (dict(n=-1), gb.EINVAL)])
def test_cache_read_int4_refuses(kw, status):
    assert read(**kw) == status


def test_nothing_to_do():
    assert rotate(rows=0, q=None, k=None, v=None, q_out=None, slots=None, positions=None) == gb.OK
    assert rotate4(rows=0, q=None, k=None, v=None, q_out=None, slots=None, positions=None) == gb.OK
    assert read(listed=0, slots=None, k=None, v=None) == gb.OK


@pytest.mark.parametrize("dim,n", [(16, 48), (64, 80), (80, 112), (96, 112), (128, 144), (144, 192), (256, 288)])
def test_int4_row_bytes(dim, n):
    assert gb.int4_row_bytes(dim) == n
    for bad in (0, -16, dim + 8, 272):
        with pytest.raises(ValueError):
            gb.int4_row_bytes(bad)


QUERY = "q dtype rows q_row q_head q_heads kv_heads dim cache slot head n ks vs".split()
QUERY_DEFAULTS = dict(q=A, dtype=1, rows=4, q_row=512, q_head=64, q_heads=8, kv_heads=2, dim=64, cache=A, slot=160, head=80, n=50,
                      ks=1.0, vs=1.0)
TAIL = "scale out lse ws ws_bytes stream".split()
TAIL_DEFAULTS = dict(scale=1.0, out=A, lse=None, ws=A, ws_bytes=1 << 30, stream=None)


def tree4(**kw):
    return call("gbtopk_tree_attention_int4", QUERY + "table cols pt_stride page lens next_n tree".split() + TAIL,
                {**QUERY_DEFAULTS, "table": A, "cols": 7, "pt_stride": 7, "page": 16, "lens": A, "next_n": 2, "tree": None,
                 **TAIL_DEFAULTS}, **kw)


def selected4(**kw):
    return call("gbtopk_selected_attention_int4", QUERY + "idx top_k idx_stride".split() + TAIL,
                {**QUERY_DEFAULTS, "idx": A, "top_k": 8, "idx_stride": 8, **TAIL_DEFAULTS}, **kw)


ATTENTION = UNITS + [
    (dict(dtype=7), gb.EINVAL), (dict(dtype=0), gb.EUNSUPPORTED), (dict(rows=-2), gb.EINVAL), (dict(q_heads=0), gb.EINVAL),
    (dict(kv_heads=3), gb.EINVAL), (dict(dim=72), gb.EUNSUPPORTED), (dict(dim=272), gb.EUNSUPPORTED), (dict(q=None), gb.EINVAL),
    (dict(cache=None), gb.EINVAL), (dict(q=A + 8), gb.EALIGN), (dict(cache=A + 8), gb.EALIGN), (dict(slot=168), gb.EALIGN),
    (dict(head=-80), gb.EINVAL), (dict(n=-1), gb.EINVAL), (dict(n=1 << 31), gb.EUNSUPPORTED), (dict(out=None), gb.EINVAL),
    (dict(out=A + 2), gb.EALIGN), (dict(lse=A + 2), gb.EALIGN), (dict(ws=None), gb.EWORKSPACE), (dict(ws=A + 16), gb.EWORKSPACE),
    (dict(ws_bytes=16), gb.EWORKSPACE)]


@pytest.mark.parametrize("kw,status", ATTENTION + [
    (dict(next_n=0), gb.EINVAL), (dict(next_n=3), gb.EINVAL), (dict(rows=130, next_n=65), gb.EUNSUPPORTED), (dict(page=0), gb.EINVAL),
    (dict(cols=-1), gb.EINVAL), (dict(pt_stride=6), gb.EINVAL), (dict(table=None), gb.EINVAL), (dict(lens=None), gb.EINVAL),
    (dict(tree=A + 4), gb.EALIGN)])
def test_tree_attention_int4_refuses(kw, status):
    assert tree4(**kw) == status


@pytest.mark.parametrize("kw,status", ATTENTION + [
    (dict(idx=None), gb.EINVAL), (dict(top_k=-1), gb.EINVAL), (dict(idx_stride=7), gb.EINVAL),
    (dict(top_k=1 << 31, idx_stride=1 << 31), gb.EUNSUPPORTED)])
def test_selected_attention_int4_refuses(kw, status):
    assert selected4(**kw) == status


@pytest.mark.parametrize("f", [tree4, selected4])
@pytest.mark.parametrize("kw", [dict(slot=208, head=96), dict(slot=176, head=80), dict(slot=64, kv_heads=1), dict(slot=(1 << 37) + 80, n=1 << 30)])
def test_attention_int4_refuses_strides_without_lines(f, kw):
    """No pitch of a row's length or more has every row on it, or too many lines."""
    assert f(**kw) == gb.EUNSUPPORTED


def prompt(**kw):
    return call("gbtopk_prompt_attention",
                "q dtype rows q_row q_head q_heads kv_heads dim k k_row k_head v v_row v_head keys cu cu_k seqs".split() + TAIL,
                dict(q=A, dtype=1, rows=100, q_row=512, q_head=64, q_heads=8, kv_heads=2, dim=64, k=A, k_row=128, k_head=64, v=A,
                     v_row=128, v_head=64, keys=100, cu=A, cu_k=None, seqs=3, **TAIL_DEFAULTS), **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), gb.EINVAL), (dict(dtype=0), gb.EUNSUPPORTED), (dict(rows=-2), gb.EINVAL), (dict(keys=-1), gb.EINVAL),
    (dict(seqs=-1), gb.EINVAL), (dict(kv_heads=3), gb.EINVAL), (dict(dim=60), gb.EUNSUPPORTED), (dict(dim=264), gb.EUNSUPPORTED),
    (dict(q=None), gb.EINVAL), (dict(k=None), gb.EINVAL), (dict(v=None), gb.EINVAL), (dict(q=A + 8), gb.EALIGN), (dict(k_row=132), gb.EALIGN),
    (dict(v_head=-64), gb.EINVAL), (dict(k_head=0), gb.EUNSUPPORTED), (dict(q_row=0), gb.EUNSUPPORTED), (dict(cu=None), gb.EINVAL),
    (dict(cu=A + 2), gb.EALIGN), (dict(cu_k=A + 1), gb.EALIGN), (dict(out=None), gb.EINVAL), (dict(out=A + 8), gb.EALIGN),
    (dict(lse=A + 2), gb.EALIGN), (dict(ws=None), gb.EWORKSPACE), (dict(ws=A + 16), gb.EWORKSPACE), (dict(ws_bytes=512), gb.EWORKSPACE),
    (dict(rows=(1 << 31) - 1), gb.EUNSUPPORTED), (dict(keys=1 << 31), gb.EUNSUPPORTED)])
def test_prompt_attention_refuses(kw, status):
    assert prompt(**kw) == status


def test_prompt_workspace():
    f = gb.gbtopk_prompt_workspace_bytes
    assert f(1000, 3, 8, 2, 64) >= 512 + 8 * (1000 // 64 + 3) and f(1000, 3, 8, 3, 64) == 0 and f(-1, 3, 8, 2, 64) == 0
    assert prompt(rows=0, q=None) == gb.OK and prompt(seqs=0) == gb.OK
