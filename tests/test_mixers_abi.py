"""Refusals of the token mixers' entry points: every bad argument is rejected on the host with
its status (fake device addresses; nothing reaches a launch), and the Python conveniences
refuse tensors that do not fit before they call the library."""
import ctypes

import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv

A = 1 << 40
MB = 1 << 20


def at(mb, off=0):
    return A + mb * MB + off


def cache(**kw):
    d = dict(k=at(0), v=at(64), k_amax=None, v_amax=None, num_pages=32, page_stride=16 * 8 * 128, token_stride=8 * 128,
             head_stride=128, page_size=16, kv_heads=8, head_dim=128, dtype=1)
    d.update(kw)
    return nv.KVCacheDesc(*[d[n] for n, _ in nv.KVCacheDesc._fields_])


def append(c=None, **kw):
    d = dict(q=at(128), k=at(160), v=at(192), src=1, T=4, heads=40, ldq=40 * 128, ldk=1024, ldv=1024, rope=at(224),
             rot=128, far=4096, inter=0, pos=at(256), slots=at(257), q_out=at(288), ldqo=40 * 128)
    d.update(kw)
    c = cache() if c is None else c
    return nv.lib().nvfp4_kv_append(d["q"], d["k"], d["v"], d["src"], d["T"], d["heads"], d["ldq"], d["ldk"], d["ldv"],
                                    d["rope"], d["rot"], d["far"], d["inter"], d["pos"], d["slots"], ctypes.byref(c),
                                    d["q_out"], d["ldqo"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(src=2), 1), (dict(k=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(rope=None), 1),
    (dict(q_out=None), 1), (dict(q=None), 1), (dict(heads=0), 1), (dict(far=-1), 1),
    (dict(rot=24), 2), (dict(rot=144), 2), (dict(rot=-16), 2), (dict(ldk=1016), 2), (dict(ldq=1024), 2),
    (dict(T=1 << 31), 2), (dict(ldv=1 << 31), 2),
    (dict(k=at(160, 8)), 3), (dict(slots=at(257, 8)), 3), (dict(ldk=1028), 3), (dict(ldqo=40 * 128 + 4), 3),
    (dict(src=0, ldk=1026), 3),
    (dict(k=at(0, 256)), 1), (dict(q_out=at(64, 256)), 1), (dict(q_out=at(128, 16)), 1), (dict(slots=at(0)), 1),
    (dict(T=0, k=None, v=None, slots=None), 0),
])
def test_append_refusals(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=96), 2), (dict(page_size=24, page_stride=24 * 1024), 2), (dict(page_size=0), 1), (dict(kv_heads=0), 1),
    (dict(dtype=0), 1), (dict(dtype=2), 1), (dict(num_pages=-1), 1), (dict(k=None), 1), (dict(v=at(0)), 1),
    (dict(num_pages=1 << 31), 2), (dict(token_stride=512), 2), (dict(page_stride=8 * 128), 2), (dict(head_stride=64), 2),
    (dict(page_stride=1 << 41), 2), (dict(token_stride=-1024), 2), (dict(page_stride=1 << 39, num_pages=1 << 30), 2),
    (dict(k=at(0, 8)), 3), (dict(page_stride=16 * 8 * 128 + 4), 3),
    (dict(dtype=2, k_amax=at(300), v_amax=at(300, 4)), 3), (dict(dtype=2, k_amax=at(300), v_amax=at(300, 16), page_stride=16 * 8 * 128 + 8), 3),
])
def test_cache_refusals(kw, status):
    assert append(c=cache(**kw)) == status
    assert attn(c=cache(**kw)) == status


def test_none_cache_is_refused():
    assert nv.lib().nvfp4_kv_append(None, at(1), at(2), 1, 1, 0, 0, 1024, 1024, None, 0, 0, 0, None, at(3), None, None, 0,
                                    None) == 1


def attn(c=None, **kw):
    d = dict(q=at(128), B=4, heads=40, ldq=40 * 128, table=at(160), ldt=32, lens=at(161), max_len=512, scale=0.1, window=0,
             out=at(192), ldo=40 * 128, lse=at(224), ws=at(256), wsb=1 << 30)
    d.update(kw)
    c = cache() if c is None else c
    return nv.lib().nvfp4_attn_decode(d["q"], d["B"], d["heads"], d["ldq"], ctypes.byref(c), d["table"], d["ldt"], d["lens"],
                                      d["max_len"], d["scale"], d["window"], d["out"], d["ldo"], d["lse"], d["ws"],
                                      d["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(heads=0), 1), (dict(heads=36), 2), (dict(max_len=-1), 1), (dict(window=-1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(max_len=513), 2), (dict(max_len=1 << 31), 2),
    (dict(window=1 << 31), 2), (dict(ldq=4096), 2), (dict(ldo=4096), 2), (dict(ldt=1 << 31), 2), (dict(B=70000), 2),
    (dict(q=None), 1), (dict(out=None), 1), (dict(lens=None), 1), (dict(table=None), 1),
    (dict(q=at(128, 8)), 3), (dict(lse=at(224, 4)), 3), (dict(lens=at(161, 4)), 3), (dict(ldo=40 * 128 + 4), 3),
    (dict(out=at(128, 64)), 1), (dict(out=at(0, 256)), 1), (dict(lse=at(161)), 1), (dict(lse=at(192)), 1),
    (dict(B=0, q=None, out=None, lens=None, table=None), 0),
])
def test_attn_refusals(kw, status):
    assert attn(**kw) == status


def test_attn_workspace_is_checked():
    """A batch whose sequences are split over workgroups needs its workspace."""
    need = nv.nvfp4_attn_decode_workspace_bytes(1, 40, 8, 128, 1 << 17, 0)
    if need == 0:
        pytest.skip("this build splits nothing")
    big = dict(c=cache(num_pages=8192, page_stride=16 * 1024, v=at(1024)), B=1, ldt=8192, max_len=1 << 17, q=at(4096),
               table=at(4100), lens=at(4104), out=at(4108), lse=at(4112), ws=at(4116))
    assert attn(**big, wsb=need - 1) == 5
    big["ws"] = None
    assert attn(**big, wsb=need) == 5
    big["ws"] = at(4116, 4)
    assert attn(**big, wsb=need) == 3
    big["ws"] = at(4096)
    assert attn(**big, wsb=need) == 1
    assert nv.nvfp4_attn_decode_workspace_bytes(-1, 40, 8, 128, 1 << 17, 0) == 0
    assert nv.nvfp4_attn_decode_workspace_bytes(1, 40, 7, 128, 1 << 17, 0) == 0


def gdn(prefill, **kw):
    d = dict(q=at(0), ldq=2048, k=at(16), ldk=2048, v=at(32), ldv=4096, g=at(64), ldg=32, beta=at(65), ldb=32, T=64, B=4,
             cu=at(66), hk=16, hv=32, dk=128, dv=128, state=at(128), n=8, index=at(67), has=at(68), scale=0.1, out=at(96),
             ldo=4096, ws=at(512), wsb=1 << 30)
    d.update(kw)
    head = [d[x] for x in ("q", "ldq", "k", "ldk", "v", "ldv", "g", "ldg", "beta", "ldb")]
    dims = [d[x] for x in ("hk", "hv", "dk", "dv", "state", "n", "index")]
    if prefill:
        return nv.lib().nvfp4_gdn_prefill(*head, d["T"], d["B"], d["cu"], *dims, d["has"], d["scale"], d["out"], d["ldo"],
                                          d["ws"], d["wsb"], None)
    return nv.lib().nvfp4_gdn_step(*head, d["B"], *dims, d["scale"], d["out"], d["ldo"], None)


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(hk=0), 1), (dict(n=-1), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(g=None), 1),
    (dict(state=None), 1), (dict(out=None), 1),
    (dict(dk=96), 2), (dict(dk=256), 2), (dict(dv=48), 2), (dict(dv=2048), 2), (dict(hk=12), 2), (dict(ldq=1024), 2),
    (dict(ldv=2048), 2), (dict(ldg=16), 2), (dict(ldb=16), 2), (dict(index=None, n=3), 2), (dict(B=70000), 2),
    (dict(n=1 << 31), 2), (dict(ldo=1 << 31), 2),
    (dict(q=at(0, 8)), 3), (dict(beta=at(65, 2)), 3), (dict(g=at(64, 1)), 3), (dict(ldk=2052), 3), (dict(state=at(128, 4)), 3),
    (dict(index=at(67, 4)), 3),
    (dict(out=at(32)), 1), (dict(state=at(16)), 1), (dict(out=at(128)), 1), (dict(state=at(64)), 1),
    (dict(B=0, q=None, state=None, out=None, cu=None), 0),
])
def test_gdn_refusals(prefill, kw, status):
    assert gdn(prefill, **kw) == status


def test_gdn_prefill_refusals():
    assert gdn(True, T=-1) == 1
    assert gdn(True, T=1 << 31) == 2
    assert gdn(True, cu=None) == 1
    assert gdn(True, cu=at(66, 4)) == 3
    assert gdn(True, out=at(66)) == 1
    need = nv.nvfp4_gdn_prefill_workspace_bytes(64, 4, 16, 32, 128, 128)
    if need:
        assert gdn(True, wsb=need - 1) == 5
        assert gdn(True, ws=None) == 5
        assert gdn(True, ws=at(512, 8)) == 3
        assert gdn(True, ws=at(96)) == 1
    assert nv.nvfp4_gdn_prefill_workspace_bytes(-1, 4, 16, 32, 128, 128) == 0


def test_accepted_calls_reach_the_runtime():
    """The calls that the tests above vary are themselves accepted: without a GPU the runtime
    refuses their launch (skipped where there is one: the addresses are fake)."""
    import os
    if os.path.exists("/dev/kfd") or torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert append() == 6 and attn() == 6 and gdn(False) == 6 and gdn(True) == 6
    inter = cache(v=at(0, 2 * 1024 * 16), page_stride=2 * 16 * 1024)     # k and v pages side by side
    assert append(c=inter) == 6 and attn(c=inter) == 6
    heads_out = cache(page_stride=16 * 128, token_stride=128, head_stride=32 * 16 * 128)
    assert append(c=heads_out) == 6
    assert append(q=None, q_out=None, heads=0) == 6 and append(rot=0, rope=None, pos=None) == 6


def test_conveniences_refuse_other_things_than_cuda_tensors():
    x = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises((AssertionError, RuntimeError)):
        nv.kv_append(x, x, None, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        nv.attn_decode(x, None, None, None, stream=7)
    with pytest.raises(AssertionError):
        nv.PagedKVCache(x.view(2, 1, 8, 128), x.view(2, 1, 8, 128))


def test_calls_larger_than_a_launch_are_refused():
    assert append(T=(1 << 22) + 1) == 2
    assert attn(B=65535, heads=72, ldq=72 * 128, ldo=72 * 128) == 2
    assert attn(max_len=(1 << 30) + 1, ldt=1 << 30) == 2
    assert nv.nvfp4_attn_decode_workspace_bytes(1, 40, 8, 128, (1 << 30) + 1, 0) == 0
    assert gdn(False, B=65535, n=1 << 17) == 2
    assert gdn(True, T=(1 << 28) + 64) == 2 and gdn(True, T=1 << 27) == 2 and gdn(True, hk=2, T=1 << 24) == 2
    assert gdn(True, B=65535, n=1 << 17) == 2
