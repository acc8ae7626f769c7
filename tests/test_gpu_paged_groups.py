"""Attention over pages with more than 64 query heads a key head on the GPU: row tiles of one token, over sequences of
several rows, one and none, in every form, against a plain 64-bit implementation."""
import math
import random

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A
from tests import serving_reference as S
from tests.test_gpu_paged import BF, i32, make, run, verify

pytestmark = pytest.mark.gpu
GROUPS = [(65, 1, 128), (71, 1, 64), (160, 2, 128), (128, 1, 64), (256, 2, 128)]
PACKS = [([0, 2], [9, 300]), ([3, 0, 0], [200, 130, 0]), ([1, 0, 1], [257, 4, 31]), ([1, 1, 1], [1, 300, 128]),
         ([0, 2, 1, 0], [20, 2, 0, 64]), ([0, 0, 5, 0, 0], [3, 0, 140, 50, 9]), ([4, 0, 0, 0], [2, 9, 9, 9])]


def wide_pool(lengths, page, seed, keys):
    """A pool and a table of at least `keys` keys for the call as a whole and for every sequence."""
    spare = (keys + page - 1) // page
    total, table = S.pool(lengths, page, random.Random(seed), spare=2 + spare)
    return total, torch.cat((table, torch.full((len(lengths), spare), 2 ** 30, dtype=torch.int32)), dim=1)


def apart(t):
    """The same pages with a gap behind each."""
    big = torch.full((t.shape[0], t.shape[1] + 1, *t.shape[2:]), math.nan, dtype=t.dtype, device=t.device)
    big[:, :-1] = t
    return big[:, :-1]


@pytest.mark.parametrize("keys", [0, 4000], ids=["small_pool", "large_pool"])
@pytest.mark.parametrize("page", [1, 2, 4, 16, 48, 128])
@pytest.mark.parametrize("heads", GROUPS, ids=str)
def test_rows_of_sequences(heads, page, keys):
    for seed, (q_lens, lengths) in enumerate(PACKS):
        verify(*run(lengths, page, heads, BF, "auto", q_lens=q_lens, seed=seed, pool=wide_pool(lengths, page, seed, keys)), lengths,
               page, q_lens, what=str(q_lens))


@pytest.mark.parametrize("keys", [0, 4000], ids=["small_pool", "large_pool"])
@pytest.mark.parametrize("page", [2, 16, 64])
@pytest.mark.parametrize("heads", GROUPS + [(8, 2, 128)], ids=str)
def test_pages_apart(heads, page, keys):
    """Decode steps without cu_q, and rows with it, over pages that do not follow one another in memory."""
    lengths = [130, 0, 64, 300]
    pool = wide_pool(lengths, page, page, keys)
    for q_lens in (None, [0, 2, 1, 1], [9, 1, 0, 2]):
        q, k, v = make(page, sum(q_lens) if q_lens else 4, pool[0], page, heads, BF)
        made, out, lse = run(lengths, page, heads, BF, "auto", q_lens=q_lens, tensors=(q, apart(k), apart(v)), pool=pool)
        verify((q, k, v, *made[3:]), out, lse, lengths, page, q_lens, what=str(q_lens))


@pytest.mark.parametrize("heads", [(128, 1, 64), (65, 1, 128)], ids=str)
def test_what_lies_behind_the_arrays_is_not_read(heads):
    """cu_q and lengths that go on, in memory, with what looks like more sequences of the same rows."""
    page, q_lens, lengths = 16, [1, 0, 2], [40, 9, 200]
    pool = wide_pool(lengths, page, 7, 0)
    q, k, v = make(7, 3, pool[0], page, heads, BF)
    table = torch.cat((pool[1], pool[1].flip(0))).cuda()
    cu, n = i32([0, 1, 1, 3, 3, 3, 0, 1, 2, 3]), i32([40, 9, 200, 16, 16, 16, 16, 16])
    see = S.see_paged(pool[1], lengths, page, q_lens)
    ref = S.attend(q, k.flatten(0, 1), v.flatten(0, 1), see, 0.1)
    ws = K.new_attention_workspace(3, 3, *heads, BF).fill_(0xFF)
    out, lse = torch.full_like(q, math.nan), torch.full(q.shape[:2], math.nan, device="cuda")
    K.kpool_attention_paged(q, k, v, table[:3], n[:3], 0.1, cu_q=cu[:4], out=out, out_lse=lse, workspace=ws)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    A.check(out, lse, ref)


def test_more_sequences_than_the_runs_take():
    heads, page = (128, 1, 64), 16
    q_lens = [(2, 0, 1)[i % 3] for i in range(8300)]
    lengths = [n + i % 5 for i, n in enumerate(q_lens)]
    (q, k, v, table, scale), out, lse = run(lengths, page, heads, BF, "auto", q_lens=q_lens, seed=8)
    pick = list(range(0, sum(q_lens), 53)) + [sum(q_lens) - 1]
    see = S.see_paged(table, lengths, page, q_lens)
    A.check(out[pick], lse[pick], S.attend(q[pick], k.flatten(0, 1), v.flatten(0, 1), [see[r] for r in pick], scale))
