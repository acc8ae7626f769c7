"""Rows of the two-row-tile form whose group size does not divide 128: the second row tile begins at row 128
of a partial result, past the rows that one tile's 128 / G tokens fill. One sequence whose keys are cut
into runs, from one token past the first tile to two full tiles; what a kernel does not write
stays NaN, so no earlier call's result can stand in for it."""
import random

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A
from tests.test_gpu_attention import BF, i32, make

pytestmark = pytest.mark.gpu
GROUPS = [3, 5, 6, 7, 12, 24, 48, 80]


def row_counts(group):
    """One token past the first row tile, one before and at two full ones, and between them, where the
    rows' number rounded up reaches least far."""
    tt = 128 // group
    return sorted({tt + 1, (3 * tt + 1) // 2, 2 * tt - 1, 2 * tt, min(256 // group, 2 * tt)} - set(range(tt + 1)))


CASES = [(g, r) for g in GROUPS for r in row_counts(g)]


def poisoned(rows, q_heads, d, kv_heads):
    out = torch.full((rows, q_heads, d), float("nan"), dtype=BF, device="cuda")
    lse = torch.full((rows, q_heads), float("nan"), device="cuda")
    ws = K.new_attention_workspace(rows, 1, q_heads, kv_heads, d, BF)
    ws.fill_(0xFF)                   # NaN wherever a partial result is read that was not written
    return dict(out=out, out_lse=lse, workspace=ws)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,rows", CASES)
def test_both_row_tiles_are_written(group, rows, d):
    heads, prefix = (2 * group, 2, d), 1500
    tokens, scale = prefix + rows, 1.0 / d ** 0.5
    q, k, v = make(group + rows, rows, tokens, heads, BF)
    ref = A.reference(q, k, v, A.see_prompt([rows], [tokens]), scale)
    cq, ck = i32([0, rows]), i32([0, tokens])
    kw = poisoned(rows, *heads[::2], heads[1])
    K.kpool_attention_prompt(q, k, v, cq, ck, scale, **kw)
    assert K.kpool_last_device_error(kw["workspace"]) == K.KPOOL_OK
    A.check(kw["out"], kw["out_lse"], ref, "prompt")
    kw = poisoned(rows, *heads[::2], heads[1])
    K.kpool_attention_tree(q, k, v, cq, ck, i32([prefix]), scale, **kw)
    A.check(kw["out"], kw["out_lse"], ref, "chain")


@pytest.mark.parametrize("group,rows", [(3, 44), (6, 24), (7, 32), (12, 20), (48, 4), (80, 2)])
def test_both_row_tiles_of_a_masked_tree_are_written(group, rows):
    heads, prefix, extent = (group, 1, 128), 4000, 4100
    bits = [A.random_tree(rows, random.Random(group))]
    q, k, v = make(group, rows, extent, heads, BF)
    kw = poisoned(rows, *heads[::2], heads[1])
    K.kpool_attention_tree(q, k, v, i32([0, rows]), i32([0, extent]), i32([prefix]), 0.08,
                           mask=A.mask_words(bits[0], (rows + 31) // 32).cuda(), **kw)
    assert K.kpool_last_device_error(kw["workspace"]) == K.KPOOL_OK
    A.check(kw["out"], kw["out_lse"], A.reference(q, k, v, A.see_tree([rows], [extent], [prefix], bits), 0.08))


def test_short_keys_of_many_key_heads():
    """Too many items for one CTA each: cut into runs although the keys are few."""
    group, kv_heads, rows = 6, 640, 24
    heads, tokens = (group * kv_heads, kv_heads, 64), 300
    q, k, v = make(5, rows, tokens, heads, BF)
    kw = poisoned(rows, *heads[::2], kv_heads)
    K.kpool_attention_prompt(q, k, v, i32([0, rows]), i32([0, tokens]), 0.125, **kw)
    assert K.kpool_last_device_error(kw["workspace"]) == K.KPOOL_OK
    A.check(kw["out"], kw["out_lse"], A.reference(q, k, v, A.see_prompt([rows], [tokens]), 0.125))
