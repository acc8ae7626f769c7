"""Refusals of the attention entry points (no GPU): every call below comes back before any pointer is used."""

import math

import pytest
import torch

from sparse_attention_kpool_gb300 import build as kbuild
from sparse_attention_kpool_gb300 import kpool as K
from tests.test_attention_devices_host import put
from tests.test_attention_host import FAKE, heads, shape

FAR = 1 << 31           # elements between tokens: a byte offset of 32 bits does not hold one


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return K.load()


def selected(lib, k, v, kernel):
    """Without a workspace: a call that is not refused for its tensors is refused for that."""
    return lib.kpool_attention_selected(heads(), k, v, FAKE, 20, FAKE, FAKE, 1, 4, 9, shape(), heads(), FAKE, None, 0,
                                        None, K.kpool_options(kernel))


@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_selected_token_strides_that_tcgen05_does_not_take(which, lib):
    k = heads(ts=FAR) if which != "v" else heads()
    v = heads(ts=FAR) if which != "k" else heads()
    assert selected(lib, k, v, K.KPOOL_SCORE_TC) == K.KPOOL_ERR_UNSUPPORTED
    assert selected(lib, k, v, K.KPOOL_SCORE_AUTO) == K.KPOOL_ERR_WORKSPACE
    assert selected(lib, k, v, K.KPOOL_SCORE_SIMT) == K.KPOOL_ERR_WORKSPACE
    assert selected(lib, heads(ts=FAR - 8), heads(ts=FAR - 8), K.KPOOL_SCORE_TC) == K.KPOOL_ERR_WORKSPACE


def test_other_operators_take_such_strides_on_tcgen05(lib):
    st = lib.kpool_attention_prompt(heads(), heads(ts=FAR), heads(ts=FAR), FAKE, FAKE, 1, 4, 9, shape(), heads(), FAKE,
                                    None, 0, None, K.kpool_options(K.KPOOL_SCORE_TC))
    assert st == K.KPOOL_ERR_WORKSPACE


@pytest.mark.parametrize("scale", [1e39, -1e39, math.inf, math.nan, 0.0, -1.0, 1e-60])
def test_scales_that_fp32_does_not_hold(scale, lib, monkeypatch):
    """The binding refuses them as the library does: out of fp32's range is not finite, or zero."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    bf, i32 = torch.bfloat16, torch.int32
    q, k = (put(0, torch.zeros((8, h, 64), dtype=bf)) for h in (4, 2))
    cu, ws = put(0, torch.zeros(2, dtype=i32)), put(0, torch.zeros(4096, dtype=torch.uint8))
    for call in (lambda: K.kpool_attention_prompt(q, k, k, cu, cu, scale, out=q, workspace=ws),
                 lambda: K.kpool_attention_tree(q, k, k, cu, cu, cu[:1], scale, out=q, workspace=ws)):
        with pytest.raises(K.KpoolError) as e:
            call()
        assert e.value.status == K.KPOOL_ERR_INVALID_ARG
