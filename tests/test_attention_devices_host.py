"""Attention calls refuse tensors that are not all on the current device (no GPU: the tensors, the library and
the devices are stand-ins): the launch goes to the current device, whatever stream it gets."""
import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K


class Placed(torch.Tensor):
    """A CPU tensor that says which device it is on (-1: the CPU)."""
    place = 0

    @property
    def is_cuda(self):
        return self.place >= 0

    def get_device(self):
        return self.place


def put(place, t):
    t = t.as_subclass(Placed)
    t.place = place
    return t


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or K.KPOOL_OK
    monkeypatch.setattr(K, "_lib", Library())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return made


def prompt(places):
    bf, i32 = torch.bfloat16, torch.int32
    names = ("q", "k", "v", "cu_q", "cu_k", "out", "lse", "workspace")
    made = (torch.zeros((8, 4, 64), dtype=bf), torch.zeros((8, 2, 64), dtype=bf), torch.zeros((8, 2, 64), dtype=bf),
            torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros((8, 4, 64), dtype=bf),
            torch.zeros((8, 4)), torch.zeros(4096, dtype=torch.uint8))
    t = {n: put(places.get(n, places.get("all", 0)), x) for n, x in zip(names, made)}
    return K.kpool_attention_prompt(t["q"], t["k"], t["v"], t["cu_q"], t["cu_k"], 0.1, out=t["out"], out_lse=t["lse"],
                                    workspace=t["workspace"])


def test_tensors_on_the_current_device_are_taken(calls):
    prompt({})
    assert calls == ["kpool_attention_prompt"]


@pytest.mark.parametrize("where", [1, -1], ids=["other_device", "cpu"])
@pytest.mark.parametrize("which", ["all", "q", "k", "v", "cu_q", "cu_k", "out", "lse", "workspace"])
def test_tensors_elsewhere_are_refused(which, where, calls):
    with pytest.raises(ValueError):
        prompt({which: where})
    assert calls == []
