"""Host-side checks of the attention entry points that need no GPU: refusals come back before
any pointer is used, and the plain reference used by the GPU tests is right on cases worked
by hand."""
import ctypes
import math

import pytest
import torch

from sparse_attention_kpool_gb300 import build as kbuild
from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A

FAKE = 0x7F0000000000      # aligned, never dereferenced: every call below is refused first
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return K.load()


def shape(hq=8, hkv=2, d=128, dtype=K.KPOOL_BF16, scale=0.1, reserved=0):
    return K.kpool_attention_shape(hq, hkv, d, dtype, scale, reserved)


def heads(data=FAKE, ts=1024, hs=128):
    return K.kpool_heads(data, ts, hs)


def prompt(lib, q=None, k=None, v=None, cu_q=FAKE, cu_k=FAKE, S=1, R=4, T=9, sh=None, out=None, lse=FAKE, ws=FAKE,
           ws_bytes=BIG, opt=None):
    return lib.kpool_attention_prompt(q or heads(), k or heads(), v or heads(), cu_q, cu_k, S, R, T, sh or shape(),
                                      out or heads(), lse, ws, ws_bytes, None, opt)


def test_struct_layouts():
    assert ctypes.sizeof(K.kpool_heads) == 24 and ctypes.sizeof(K.kpool_attention_shape) == 24


BAD_SHAPES = [dict(hq=7), dict(hq=0), dict(hkv=0), dict(d=0), dict(d=12), dict(d=-8), dict(dtype=2),
              dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(reserved=1)]


@pytest.mark.parametrize("bad", BAD_SHAPES, ids=str)
def test_bad_shapes(lib, bad):
    assert prompt(lib, sh=shape(**bad)) == K.KPOOL_ERR_INVALID_ARG
    assert lib.kpool_attention_workspace_bytes(4, 1, shape(**bad)) == 0


@pytest.mark.parametrize("far", [dict(d=264), dict(hq=129, hkv=1), dict(hq=8192, hkv=128)], ids=str)
def test_unsupported_shapes(lib, far):
    assert prompt(lib, sh=shape(**far)) == K.KPOOL_ERR_UNSUPPORTED


BAD_HEADS = [dict(data=None), dict(data=FAKE + 8), dict(ts=64), dict(hs=64), dict(ts=0), dict(hs=-128), dict(ts=1025),
             dict(hs=132), dict(ts=1 << 40)]


@pytest.mark.parametrize("bad", BAD_HEADS, ids=str)
@pytest.mark.parametrize("which", ["q", "k", "v", "out"])
def test_bad_tensors(lib, bad, which):
    assert prompt(lib, **{which: heads(**bad)}) == K.KPOOL_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(R=-1), dict(T=-1), dict(S=-1), dict(S=0), dict(R=1 << 31), dict(T=1 << 31),
                                 dict(cu_q=None), dict(cu_k=None), dict(cu_q=FAKE + 2), dict(cu_k=FAKE + 1),
                                 dict(lse=FAKE + 2)], ids=str)
def test_bad_arguments(lib, bad):
    assert prompt(lib, **bad) == K.KPOOL_ERR_INVALID_ARG


def test_bad_workspace(lib):
    assert prompt(lib, ws=None) == K.KPOOL_ERR_WORKSPACE
    assert prompt(lib, ws=FAKE + 128) == K.KPOOL_ERR_WORKSPACE
    n = lib.kpool_attention_workspace_bytes(4, 1, shape())
    assert n >= 256 and prompt(lib, ws_bytes=n - 1) == K.KPOOL_ERR_WORKSPACE


def test_bad_options(lib):
    for opt in (K.kpool_options(3), K.kpool_options(-1), K.kpool_options(0, 1), K.kpool_options(0, 0, None, 1),
                K.kpool_options(0, 0, None, 0, 0, 1), K.kpool_options(0, 0, None, 0, 0, 0, 1)):
        assert prompt(lib, opt=opt) == K.KPOOL_ERR_INVALID_ARG
    assert prompt(lib, sh=shape(dtype=K.KPOOL_F32), opt=K.kpool_options(K.KPOOL_SCORE_TC)) == K.KPOOL_ERR_UNSUPPORTED


def test_no_rows_is_a_no_op(lib):
    assert prompt(lib, R=0, cu_q=None, ws=None) == K.KPOOL_OK


def tree(lib, prefix=FAKE, mask=FAKE, words=1, cu_q=FAKE):
    return lib.kpool_attention_tree(heads(), heads(), heads(), cu_q, FAKE, prefix, mask, words, 1, 4, 9, shape(),
                                    heads(), FAKE, FAKE, 0, None, None)


def test_tree_refusals(lib):
    assert tree(lib) == K.KPOOL_ERR_WORKSPACE
    for bad in (dict(prefix=None), dict(prefix=FAKE + 2), dict(mask=None), dict(words=0), dict(words=-1),
                dict(mask=FAKE + 1), dict(cu_q=None), dict(words=1 << 21)):
        assert tree(lib, **bad) == K.KPOOL_ERR_INVALID_ARG
    assert tree(lib, mask=None, words=0) == K.KPOOL_ERR_WORKSPACE


def selected(lib, ids=FAKE, width=20, row_seq=FAKE, R=4, T=9):
    return lib.kpool_attention_selected(heads(), heads(), heads(), ids, width, row_seq, FAKE, 1, R, T, shape(), heads(),
                                        FAKE, FAKE, 0, None, None)


def test_selected_refusals(lib):
    assert selected(lib) == K.KPOOL_ERR_WORKSPACE
    for bad in (dict(ids=None), dict(ids=FAKE + 2), dict(width=-1), dict(row_seq=FAKE + 1), dict(row_seq=None)):
        assert selected(lib, **bad) == K.KPOOL_ERR_INVALID_ARG
    assert selected(lib, row_seq=None, R=9) == K.KPOOL_ERR_WORKSPACE


def test_binding_refusals():
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    k = torch.zeros((9, 2, 128), dtype=torch.bfloat16)
    c = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        K.kpool_attention_prompt(q, k, k[:, :1], c, c, 0.1)
    with pytest.raises(TypeError):
        K.kpool_attention_prompt(q, k.float(), k, c, c, 0.1)
    with pytest.raises(ValueError):
        K.kpool_attention_prompt(q, k, k, c, c[:1], 0.1)
    with pytest.raises(TypeError):
        K.kpool_attention_prompt(q.half(), k.half(), k.half(), c, c, 0.1, workspace=q)
    with pytest.raises(TypeError):
        K.kpool_attention_prompt(q, k, k, c, c, 0.1, out=q[:2], workspace=q)
    with pytest.raises(ValueError):
        K.kpool_attention_tree(q, k, k, c, c, c, 0.1)
    with pytest.raises(ValueError):
        K.kpool_attention_tree(q, k, k, c, c, c[:1], 0.1, mask=torch.zeros((4, 0), dtype=torch.int32))
    with pytest.raises(ValueError):
        K.kpool_attention_selected(q, k, k, torch.zeros((3, 5), dtype=torch.int32), c, 0.1)


def test_reference_by_hand():
    """Two keys with scores ln 3 and 0: weights 3/4 and 1/4; an empty row; a key named twice."""
    q = torch.tensor([[[1.0, 0.0]]] * 3)
    k = torch.tensor([[[math.log(3.0), 5.0]], [[0.0, -2.0]]])
    v = torch.tensor([[[4.0, 0.0]], [[0.0, 8.0]]])
    out, lse, tol, _ = A.reference(q, k, v, [torch.tensor([0, 1]), torch.tensor([], dtype=torch.int64),
                                             torch.tensor([0, 1, 1])], 1.0)
    assert torch.allclose(out[:, 0], torch.tensor([[3.0, 2.0], [0.0, 0.0], [2.4, 3.2]], dtype=torch.float64), atol=1e-6)
    assert torch.allclose(lse[[0, 2], 0], torch.tensor([math.log(4.0), math.log(5.0)], dtype=torch.float64), atol=1e-6)
    assert lse[1, 0] == -math.inf
    assert (tol[0] < 1e-4).all() and (tol[0] > 0).all()


def test_visible_sets_by_hand():
    assert [x.tolist() for x in A.see_prompt([2, 3], [3, 1])] == [[0, 1], [0, 1, 2], [], [], [3]]
    assert [x.tolist() for x in A.see_tree([2], [9], [3], [[0b10, 0b11]])] == [[0, 1, 2, 4], [0, 1, 2, 3, 4]]
    assert [x.tolist() for x in A.see_tree([2], [9], [1], None)] == [[0, 1], [0, 1, 2]]
    assert A.mask_words([1 << 31 | 1, 1 << 32], 2).tolist() == [[-2 ** 31 + 1, 0], [0, 1]]
