"""What a call on a named stream allocates comes from that stream's memory (no GPU: the library, the streams
and the allocations are stand-ins that write down what they are asked for)."""
import contextlib

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K

SIDE = 0x5EED0          # the handle of "another stream"


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on the GPU and remembers the streams recorded on it."""
    is_cuda = True

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream]


class Library:
    """Every entry point succeeds; sizes are 4096."""

    def __getattr__(self, name):
        return (lambda *a: 4096) if name.endswith("_bytes") else (lambda *a: K.KPOOL_OK)


@pytest.fixture
def world(monkeypatch):
    seen = {"stream": ["here"], "made": []}
    empty = torch.empty

    def make(*a, **kw):
        t = empty(*a, **kw).as_subclass(OnDevice)
        seen["made"].append((t, seen["stream"][-1]))
        return t

    @contextlib.contextmanager
    def on(stream):
        seen["stream"].append(stream)
        yield
        seen["stream"].pop()
    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: seen["stream"][-1])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, *a: handle)
    monkeypatch.setattr(K, "_lib", Library())
    return seen


def dev(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


def ints(*shape):
    return dev(*shape, dtype=torch.int32)


def f32(*shape):
    return dev(*shape, dtype=torch.float32)


INDEX = lambda: (dev(8, 2, 64), dev(8, 64), f32(8, 2), ints(2))  # noqa: E731
HEADS = lambda: (dev(8, 4, 64), dev(8, 2, 64), dev(8, 2, 64))  # noqa: E731
# call -> tensors it makes: outputs and a workspace
CALLS = {
    "select": (lambda **kw: K.kpool_select_ex(*INDEX(), 4, 8, 1.0, return_scores=True, **kw), 4),
    "static_scratch": (lambda **kw: K.kpool_select_static_scratch(*INDEX(), 4, 8, 1.0, return_scores=True, **kw), 3),
    "pooled": (lambda **kw: K.kpool_select_pooled(*INDEX(), 4, 8, 1.0, return_scores=True, **kw), 4),
    "rows": (lambda **kw: K.kpool_select_rows(dev(3, 2, 64), f32(3, 2), ints(3), ints(3), dev(2, 64), ints(2), 8, 4, 8,
                                              1.0, return_scores=True, **kw), 4),
    "pool_keys": (lambda **kw: K.kpool_pool_keys(dev(8, 64), ints(2), 4, **kw), 2),
    "pool_keys_gated": (lambda **kw: K.kpool_pool_keys_gated(dev(8, 64), f32(8, 64), f32(4, 64), ints(2), 4, **kw), 2),
    "expand": (lambda **kw: K.kpool_expand(ints(8, 2), ints(2), 4, 8, **kw), 1),
    "index_scores": (lambda **kw: K.kpool_index_scores(*INDEX(), 4, 1.0, **kw), 2),
    "prompt": (lambda **kw: K.kpool_attention_prompt(*HEADS(), ints(2), ints(2), 1.0, return_lse=True, **kw), 3),
    "tree": (lambda **kw: K.kpool_attention_tree(*HEADS(), ints(2), ints(2), ints(1), 1.0, return_lse=True, **kw), 3),
    "selected": (lambda **kw: K.kpool_attention_selected(*HEADS(), ints(8, 5), ints(2), 1.0, return_lse=True, **kw), 3),
}


@pytest.mark.parametrize("handle,stream", [(SIDE, SIDE), (0, "default")], ids=["side", "default"])
@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_another_stream_allocates_there(name, handle, stream, world):
    call, count = CALLS[name]
    got = call(stream=handle)
    assert [s for _, s in world["made"]] == [stream] * count
    got = [t for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
    for t, _ in world["made"]:
        # what the caller gets is used on its own stream, too; a workspace is not
        back = any(t.data_ptr() == x.data_ptr() for x in got)
        assert getattr(t, "recorded", []) == (["here"] if back else [])
    assert world["stream"] == ["here"]


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_the_current_stream_allocates_as_ever(name, world, monkeypatch):
    monkeypatch.setattr(K, "_stream", lambda s: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    call, count = CALLS[name]
    call()
    assert [s for _, s in world["made"]] == ["here"] * count
    assert not any(hasattr(t, "recorded") for t, _ in world["made"])
