"""Refusals of the entry points for drafted tokens: every bad argument is rejected on the host with
its status (fake device addresses; nothing reaches a launch), and the Python conveniences refuse
tensors that do not fit before they call the library."""
import ctypes
import inspect
import os

import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from test_mixers_abi import at, cache


def norm(c=None, **kw):
    d = dict(q=at(128), k=at(160), v=at(192), src=1, T=4, heads=40, ldq=40 * 128, ldk=1024, ldv=1024, qn=at(320), kn=at(321),
             eps=1e-6, rope=at(224), rot=128, far=4096, inter=0, pos=at(256), slots=at(257), q_out=at(288), ldqo=40 * 128)
    d.update(kw)
    c = cache() if c is None else c
    return nv.lib().nvfp4_kv_append_norm(d["q"], d["k"], d["v"], d["src"], d["T"], d["heads"], d["ldq"], d["ldk"], d["ldv"],
                                         d["qn"], d["kn"], d["eps"], d["rope"], d["rot"], d["far"], d["inter"], d["pos"],
                                         d["slots"], ctypes.byref(c), d["q_out"], d["ldqo"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(q=None, q_out=None, heads=0), 1),
    (dict(qn=at(320, 8)), 3), (dict(kn=at(320, 4)), 3), (dict(qn=at(0)), 1), (dict(kn=at(288)), 1), (dict(kn=at(64, 512)), 1),
    (dict(T=-1), 1), (dict(k=None), 1), (dict(slots=None), 1), (dict(rot=24), 2), (dict(ldq=1024), 2), (dict(k=at(160, 8)), 3),
    (dict(q_out=at(128, 16)), 1), (dict(T=(1 << 22) + 1), 2), (dict(T=0, k=None, v=None, slots=None), 0),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


def tree(c=None, **kw):
    d = dict(q=at(128), B=4, W=8, heads=40, ldq=40 * 128, table=at(160), ldt=33, lens=at(161), parents=at(162), max_len=512,
             scale=0.1, window=0, out=at(192), ldo=40 * 128, lse=at(224), ws=at(256), wsb=1 << 30)
    d.update(kw)
    c = cache() if c is None else c
    return nv.lib().nvfp4_attn_tree(d["q"], d["B"], d["W"], d["heads"], d["ldq"], ctypes.byref(c), d["table"], d["ldt"],
                                    d["lens"], d["parents"], d["max_len"], d["scale"], d["window"], d["out"], d["ldo"],
                                    d["lse"], d["ws"], d["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(W=0), 1), (dict(heads=0), 1), (dict(max_len=-1), 1), (dict(window=-1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(W=65), 2), (dict(heads=36), 2), (dict(max_len=521), 2), (dict(ldt=32), 2), (dict(max_len=(1 << 30) + 1, ldt=1 << 30), 2),
    (dict(window=1 << 31), 2), (dict(ldq=4096), 2), (dict(ldo=4096), 2), (dict(ldt=1 << 31), 2), (dict(B=70000), 2),
    (dict(B=65535), 2), (dict(B=1639, W=64), 2),
    (dict(q=None), 1), (dict(out=None), 1), (dict(lens=None), 1), (dict(table=None), 1),
    (dict(q=at(128, 8)), 3), (dict(lse=at(224, 4)), 3), (dict(lens=at(161, 4)), 3), (dict(parents=at(162, 4)), 3),
    (dict(ldo=40 * 128 + 4), 3), (dict(ldq=40 * 128 + 4), 3),
    (dict(out=at(128, 64)), 1), (dict(out=at(0, 256)), 1), (dict(lse=at(161)), 1), (dict(lse=at(162)), 1), (dict(lse=at(192)), 1),
    (dict(B=0, q=None, out=None, lens=None, table=None), 0),
])
def test_tree_refusals(kw, status):
    assert tree(**kw) == status


def test_tree_workspace_is_checked():
    need = nv.nvfp4_attn_tree_workspace_bytes(1, 8, 40, 8, 128, 1 << 17, 0)
    assert need > 0
    big = dict(c=cache(num_pages=8192, page_stride=16 * 1024, v=at(1024)), B=1, ldt=8193, max_len=1 << 17, q=at(4096),
               table=at(4100), lens=at(4104), parents=at(4105), out=at(4108), lse=at(4112), ws=at(4116))
    assert tree(**big, wsb=need - 1) == 5
    big["ws"] = None
    assert tree(**big, wsb=need) == 5
    big["ws"] = at(4116, 4)
    assert tree(**big, wsb=need) == 3
    big["ws"] = at(4096)
    assert tree(**big, wsb=need) == 1
    for bad in ((-1, 8, 40, 8, 128, 1 << 17, 0), (1, 0, 40, 8, 128, 1 << 17, 0), (1, 65, 40, 8, 128, 1 << 17, 0),
                (1, 8, 40, 7, 128, 1 << 17, 0), (1, 8, 40, 8, 128, (1 << 30) + 1, 0), (1, 8, 40, 8, 128, 64, -1)):
        assert nv.nvfp4_attn_tree_workspace_bytes(*bad) == 0


def verify(**kw):
    d = dict(logits=at(0), B=4, W=8, V=32000, ld=32000, draft=None, ldd=0, drafts=at(64), parents=at(65), temp=at(66), u=at(67),
             tokens=at(68), path=at(69), counts=at(70), ws=at(71), wsb=1 << 30)
    d.update(kw)
    return nv.lib().nvfp4_verify_drafts(d["logits"], d["B"], d["W"], d["V"], d["ld"], d["draft"], d["ldd"], d["drafts"],
                                        d["parents"], d["temp"], d["u"], d["tokens"], d["path"], d["counts"], d["ws"], d["wsb"],
                                        None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(W=0), 1), (dict(V=0), 1), (dict(logits=None), 1), (dict(drafts=None), 1), (dict(tokens=None), 1),
    (dict(path=None), 1), (dict(counts=None), 1), (dict(u=None), 1),
    (dict(W=65), 2), (dict(B=65536), 2), (dict(ld=31999), 2), (dict(draft=at(200), ldd=100), 2), (dict(V=(1 << 31) - 1, ld=(1 << 31) - 1), 2),
    (dict(ld=1 << 31), 2), (dict(B=65535, W=64, V=8193, ld=8193), 2),
    (dict(ws=None), 5), (dict(wsb=16), 5), (dict(ws=at(71, 8)), 3), (dict(logits=at(0, 4)), 3), (dict(drafts=at(64, 8)), 3),
    (dict(parents=at(65, 4)), 3), (dict(temp=at(66, 4)), 3), (dict(u=at(67, 4)), 3), (dict(tokens=at(68, 8)), 3),
    (dict(path=at(69, 4)), 3), (dict(counts=at(70, 4)), 3), (dict(draft=at(200, 4), ldd=32000), 3),
    (dict(tokens=at(0, 16)), 1), (dict(path=at(64)), 1), (dict(counts=at(67)), 1), (dict(ws=at(3)), 1), (dict(path=at(68)), 1),
    (dict(B=0, logits=None, drafts=None, tokens=None, path=None, counts=None, ws=None), 0),
])
def test_verify_refusals(kw, status):
    assert verify(**kw) == status


def test_verify_workspace_queries():
    plain, drawn = (nv.nvfp4_verify_drafts_workspace_bytes(4, 8, 32000, x) for x in (0, 1))
    assert 0 < plain < drawn and verify(draft=at(200), ldd=32000, wsb=drawn - 1) == 5
    for bad in ((0, 8, 32000, 0), (4, 0, 32000, 0), (4, 65, 32000, 0), (4, 8, 0, 0), (4, 8, 1 << 31, 0)):
        assert nv.nvfp4_verify_drafts_workspace_bytes(*bad) == 0


def layers(*cs):
    return (nv.KVCacheDesc * len(cs))(*cs), len(cs)


def compact(cs=None, n=None, **kw):
    d = dict(table=at(160), ldt=32, B=4, W=8, lens=at(161), path=at(162), counts=at(163))
    d.update(kw)
    arr, m = layers(*([cache()] if cs is None else cs))
    return nv.lib().nvfp4_kv_compact(arr, m if n is None else n, d["table"], d["ldt"], d["B"], d["W"], d["lens"], d["path"],
                                     d["counts"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), 1), (dict(n=-1), 1), (dict(B=-1), 1), (dict(W=0), 1), (dict(ldt=-1), 1), (dict(lens=None), 1), (dict(path=None), 1),
    (dict(counts=None), 1), (dict(table=None), 1), (dict(W=65), 2), (dict(B=65536), 2), (dict(ldt=1 << 31), 2),
    (dict(table=at(160, 4)), 3), (dict(lens=at(161, 8)), 3), (dict(path=at(162, 4)), 3), (dict(counts=at(163, 4)), 3),
    (dict(path=at(0, 64)), 1), (dict(table=at(64)), 1), (dict(B=0, lens=None, path=None, counts=None, table=None), 0),
])
def test_compact_refusals(kw, status):
    assert compact(**kw) == status


def copy(cs=None, n=3, src=at(160), dst=at(161), m=None):
    arr, k = layers(*([cache()] if cs is None else cs))
    return nv.lib().nvfp4_kv_copy_pages(arr, k if m is None else m, src, dst, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(src=None), 1), (dict(dst=None), 1), (dict(m=0), 1), (dict(n=1 << 31), 2), (dict(n=1 << 21), 2),
    (dict(src=at(160, 4)), 3), (dict(dst=at(161, 8)), 3), (dict(dst=at(0)), 1), (dict(src=at(64, 1024)), 1),
    (dict(n=0, src=None, dst=None), 0),
])
def test_copy_refusals(kw, status):
    assert copy(**kw) == status


@pytest.mark.parametrize("call", [compact, copy])
def test_layers_are_checked(call):
    far = cache(k=at(500), v=at(564))
    assert call(cs=[cache(), cache()]) == 1                                     # the same cache twice
    assert call(cs=[cache(), cache(k=at(64), v=at(500))]) == 1                  # one's k is the other's v
    assert call(cs=[cache(), cache(k=at(500), v=at(0))]) == 1
    assert call(cs=[cache(), far, cache(k=at(600), v=at(564))]) == 1
    for other in (dict(num_pages=31), dict(page_stride=32 * 1024), dict(head_dim=64), dict(kv_heads=4), dict(page_size=32, page_stride=32 * 1024),
                  dict(dtype=2, k_amax=at(300), v_amax=at(301))):
        assert call(cs=[cache(), cache(**{**dict(k=at(500), v=at(564)), **other})]) == 2
    assert call(cs=[cache(), cache(k=at(500, 8), v=at(564))]) == 3
    assert call(cs=[cache(), cache(k=None, v=at(564))]) == 1
    many = [cache(k=at(1000 + 2 * i), v=at(1001 + 2 * i)) for i in range(65)]
    assert call(cs=many) == 2
    lib = nv.lib()
    assert lib.nvfp4_kv_compact(None, 1, at(160), 32, 4, 8, at(161), at(162), at(163), None) == 1
    assert lib.nvfp4_kv_copy_pages(None, 1, at(160), at(161), 1, None) == 1


def test_accepted_calls_reach_the_runtime():
    """The calls that the tests above vary are themselves accepted: without a GPU the runtime
    refuses their launch (skipped where there is one: the addresses are fake)."""
    if os.path.exists("/dev/kfd") or torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert norm() == 6 and norm(qn=None) == 6 and norm(kn=None, qn=None) == 6 and norm(q=None, q_out=None, heads=0, qn=None) == 6
    assert tree() == 6 and tree(parents=None) == 6 and tree(W=64, ldt=36) == 6 and tree(W=1, max_len=0, ldt=1) == 6
    assert verify() == 6 and verify(draft=at(200), ldd=32001) == 6 and verify(temp=None, u=None, parents=None) == 6
    assert verify(temp=None, u=None, draft=at(200, 4), ldd=0) == 6               # the greedy rule asks no draft model
    apart = [cache(k=at(1000 + 2 * i), v=at(1001 + 2 * i)) for i in range(64)]
    assert compact() == 6 and compact(cs=apart) == 6 and copy() == 6 and copy(cs=apart) == 6
    # layers interleaved in one allocation, page by page
    inter = [cache(k=at(0, (2 * i) * 32768), v=at(0, (2 * i + 1) * 32768), page_stride=8 * 16 * 1024) for i in range(4)]
    assert compact(cs=inter) == 6 and copy(cs=inter) == 6
    clash = inter[:3] + [cache(k=at(0, 5 * 32768), v=at(0, 7 * 32768), page_stride=8 * 16 * 1024)]
    assert compact(cs=clash) == 1 and copy(cs=clash) == 1


@pytest.mark.parametrize("fn", [nv.attn_tree, nv.verify_drafts, nv.kv_compact, nv.kv_copy_pages])
def test_every_argument_can_be_given_by_name(fn):
    names = [p.name for p in inspect.signature(fn).parameters.values() if p.default is p.empty]
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(AssertionError, match="cuda tensor"):
        fn(**{n: x for n in names})
    with pytest.raises(TypeError, match=names[0]):
        fn(None, **{n: x for n in names[1:]})
    with pytest.raises(TypeError):
        fn(x, *([x] * (len(names) - 1)), stream=7)
