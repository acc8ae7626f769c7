"""What a rotary, paged or latent call on a named stream allocates comes from that stream's memory (no GPU: stand-ins)."""
import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests.test_stream_memory_host import SIDE, dev, ints, world  # noqa: F401 (a fixture)


def table():
    return dev(32, dtype=torch.int64)


PAGED = lambda: (dev(3, 4, 64), dev(5, 16, 2, 64), dev(5, 16, 2, 64), ints(3, 4), ints(3))  # noqa: E731
PROMPT = lambda: (dev(3, 4, 48), dev(5, 4, 32), dev(5, 16), dev(5, 4, 64), ints(2), ints(2))  # noqa: E731
# call -> tensors it makes: outputs and a workspace
CALLS = {
    "paged": (lambda **kw: K.kpool_attention_paged(*PAGED(), 1.0, return_lse=True, **kw), 3),
    "latent": (lambda **kw: K.kpool_attention_latent(dev(3, 4, 80), dev(5, 16, 80), ints(3, 4), ints(3), 64, 1.0,
                                                     return_lse=True, **kw), 3),
    "latent_prompt": (lambda **kw: K.kpool_attention_latent_prompt(*PROMPT(), 1.0, return_lse=True, **kw), 3),
    "rotary": (lambda **kw: K.kpool_rotary(dev(3, 4, 64), ints(3), table(), k=dev(3, 1, 64), **kw), 2),
}


@pytest.mark.parametrize("handle,stream", [(SIDE, SIDE), (0, "default")], ids=["side", "default"])
@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_another_stream_allocates_there(name, handle, stream, world):  # noqa: F811
    call, count = CALLS[name]
    got = [t for t in call(stream=handle) if t is not None]
    assert [s for _, s in world["made"]] == [stream] * count
    for t, _ in world["made"]:
        back = any(t.data_ptr() == x.data_ptr() for x in got)
        assert getattr(t, "recorded", []) == (["here"] if back else [])
    assert world["stream"] == ["here"]


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_the_current_stream_allocates_as_ever(name, world, monkeypatch):  # noqa: F811
    monkeypatch.setattr(K, "_stream", lambda s: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    call, count = CALLS[name]
    call()
    assert [s for _, s in world["made"]] == ["here"] * count
    assert not any(hasattr(t, "recorded") for t, _ in world["made"])
