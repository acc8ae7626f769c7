"""Refusals of the attention entry points (no GPU): every call below comes back before any pointer is used."""

import pytest

from sparse_attention_kpool_gb300 import build as kbuild
from sparse_attention_kpool_gb300 import kpool as K
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
