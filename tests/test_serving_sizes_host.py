"""Sizes past 31 bits: the binding refuses what the library's arguments do not hold, instead of passing their low bits (no
GPU: tensors without memory, the library is a stand-in)."""
import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests.test_attention_devices_host import calls, put  # noqa: F401 (a fixture)

BF, I32 = torch.bfloat16, torch.int32
FAR = 2 ** 32 + 3


def here(*shape, dtype=BF):
    return put(0, torch.empty(shape, dtype=dtype, device="meta"))


def paged(pages=5, size=16, columns=4):
    kv = [here(pages, size, 2, 64) for _ in range(2)]
    K.kpool_attention_paged(here(3, 4, 64), *kv, here(3, columns, dtype=I32), here(3, dtype=I32), 0.1, out=here(3, 4, 64),
                            workspace=here(64, dtype=torch.uint8))


def latent(pages=5, size=16, columns=4, width=9):
    K.kpool_attention_latent(here(3, 4, 80), here(pages, size, 80), here(3, columns, dtype=I32), here(3, dtype=I32), 64, 0.1,
                             token_ids=here(3, width, dtype=I32), out=here(3, 4, 64), workspace=here(64, dtype=torch.uint8))


def many_sequences(n):
    K.kpool_attention_paged(here(3, 4, 64), here(5, 16, 2, 64), here(5, 16, 2, 64), here(n, 4, dtype=I32), here(n, dtype=I32), 0.1,
                            cu_q=here(n + 1, dtype=I32), out=here(3, 4, 64), workspace=here(64, dtype=torch.uint8))


def many_sequences_latent(n):
    K.kpool_attention_latent(here(3, 4, 80), here(5, 16, 80), here(n, 4, dtype=I32), here(n, dtype=I32), 64, 0.1,
                             row_seq=here(3, dtype=I32), out=here(3, 4, 64), workspace=here(64, dtype=torch.uint8))


def many_prompts(n):
    cu = here(n + 1, dtype=I32)
    K.kpool_attention_latent_prompt(here(3, 4, 48), here(5, 4, 32), here(5, 16), here(5, 4, 64), cu, cu, 0.1, out=here(3, 4, 64),
                                    workspace=here(64, dtype=torch.uint8))


CASES = [(paged, n) for n in ("pages", "size", "columns")] + [(latent, n) for n in ("pages", "size", "columns", "width")] + \
    [(f, "n") for f in (many_sequences, many_sequences_latent, many_prompts)]


@pytest.mark.parametrize("call,name", CASES, ids=lambda x: x if isinstance(x, str) else x.__name__)
def test_sizes_past_31_bits_are_refused(call, name, calls):  # noqa: F811
    call(**{name: 3})
    assert len(calls) == 1
    with pytest.raises(ValueError):
        call(**{name: FAR})
    assert len(calls) == 1
