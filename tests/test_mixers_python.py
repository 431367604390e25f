"""The mixers' Python layer on the CPU: what a caller may rely on before a call reaches the
library (which needs a GPU)."""
import inspect
import weakref

import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv


@pytest.mark.parametrize("name", ["k", "v", "k_amax", "v_amax"])
def test_a_caches_tensors_cannot_be_replaced(name):
    """The descriptor holds their addresses, so another tensor in a tensor's place is refused."""
    cache = nv.PagedKVCache.__new__(nv.PagedKVCache)       # (its constructor wants cuda tensors)
    with pytest.raises(AttributeError):
        setattr(cache, name, torch.zeros(1))


def test_a_captured_calls_scratch_outlives_growth(monkeypatch):
    """A graph that was captured with a small Workspace writes into that buffer at every replay:
    a larger call after it must not give the buffer back to the allocator."""
    capturing = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    ws = nv.Workspace("cpu")
    eager = weakref.ref(ws.get(64)[0])
    assert ws.get(128)[1] == 128 and eager() is None        # nobody has it: freed
    capturing[0] = True
    first = weakref.ref(ws.get(100)[0])
    capturing[0] = False
    assert ws.get(100)[0] is first() and ws.get(0) == (None, 0)
    assert ws.get(4096)[1] == 4096
    assert first() is not None
    second = weakref.ref(ws.get(4096)[0])
    ws.get(8192)
    assert second() is None
    kept = first().data_ptr()
    del ws
    assert kept and first() is None


def test_a_workspace_of_another_device_is_refused(monkeypatch):
    """Its address would be another device's, or the host's, to the kernel."""
    class OnGpu:
        device = "cuda:0"

        def get_device(self):
            return 0

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    ws = nv.Workspace("cpu")
    with pytest.raises(AssertionError, match="workspace"):
        nv._scratch(ws, OnGpu(), 64)
    assert nv._scratch(ws, OnGpu(), 0) == (None, 0)        # nothing is needed
    buf, n = nv._scratch(None, torch.zeros(1), 64)
    assert buf.numel() == n == 64


def test_growth_on_another_stream_waits_for_it(monkeypatch):
    """A buffer allocated on one stream and last used on another goes back to the allocator
    together with the stream of the call that grows the Workspace."""
    class Buffer:
        is_cuda, device, streams = True, "cuda:0", []

        def numel(self):
            return 64

        def record_stream(self, stream):
            self.streams.append(stream)

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: ("stream of", device))
    ws = nv.Workspace("cpu")
    ws.buf = old = Buffer()
    assert ws.get(64) == (old, 64) and old.streams == []
    ws.get(65)
    assert old.streams == [("stream of", "cuda:0")]


@pytest.mark.parametrize("fn", [nv.kv_append, nv.attn_decode, nv.gdn_step, nv.gdn_prefill])
def test_every_argument_can_be_given_by_name(fn):
    """By the names that the signature shows, the first tensor's too: with tensors on the CPU the
    call gets as far as the check that refuses them."""
    names = [p.name for p in inspect.signature(fn).parameters.values() if p.default is p.empty]
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(AssertionError, match="cuda tensor"):
        fn(**{n: x for n in names})
    with pytest.raises(AssertionError, match="cuda tensor"):
        fn(x, **{n: x for n in names[1:]})
    with pytest.raises(TypeError, match=names[0]):
        fn(**{n: x for n in names[1:]})
    with pytest.raises(TypeError, match=names[0]):
        fn(None, **{n: x for n in names[1:]})


def test_a_library_of_an_earlier_build_is_named(monkeypatch):
    """A library without the mixers has the same version number: loading it says what is wrong."""
    class Function:
        pass

    class Earlier:
        def __getattr__(self, name):
            if name.startswith(("nvfp4_gdn", "nvfp4_attn", "nvfp4_kv_append")):
                raise AttributeError(f"undefined symbol: {name}")
            return Function()

    nv.lib()
    monkeypatch.setattr(nv, "_LIB", None)
    monkeypatch.setattr(nv.ctypes, "CDLL", lambda path: Earlier())
    with pytest.raises(ImportError, match="earlier build.*nvfp4_kv_append"):
        nv.lib()
