"""What a pool and a page table could hold does not change how a paged call works: the same rows in an exact and in a wide
pool, and calls of many long rows, which are cut by the lengths, against a plain 64-bit implementation."""
import math
import random

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A
from tests import serving_reference as S
from tests.test_gpu_paged import BF, i32, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [64, 2])
@pytest.mark.parametrize("n", [256, 100])
def test_many_short_prompts_under_a_wide_table(n, page):
    """Bit for bit what a table of their own size gives: the same work on the same CTAs."""
    count, wide, heads = 64 if n == 256 else 128, 16384, (32, 2, 64)
    lengths = [n] * count
    total, table = S.pool(lengths, page, random.Random(n))
    q, k, v = make(n, n * count, total, page, heads, BF)
    _, want, wlse = run(lengths, page, heads, BF, "auto", q_lens=lengths, tensors=(q, k, v), pool=(total, table))
    big = 8192 * count // page + 1
    kb, vb = (torch.zeros((big, *t.shape[1:]), dtype=BF, device="cuda") for t in (k, v))
    kb[:total], vb[:total] = k, v
    broad = torch.full((count, wide // page), 2 ** 30, dtype=torch.int32)
    broad[:, :table.shape[1]] = table
    _, out, lse = run(lengths, page, heads, BF, "auto", q_lens=lengths, tensors=(q, kb, vb), pool=(big, broad))
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("heads", [(64, 4, 64), (32, 8, 128), (128, 1, 128)], ids=str)
@pytest.mark.parametrize("q_lens,lengths", [
    ([1024] * 4, [9000] * 4), ([2000, 0, 1030, 1, 1500], [12000, 9000, 9500, 8200, 8192]), ([3000, 900], [30000, 900]),
    ([1600, 40, 0, 1600], [9000, 20, 16000, 16000]), ([4100], [4096])], ids=str)
def test_long_sequences(q_lens, lengths, heads):
    """Above and below the means of the rule, empty sequences between others, more rows than keys; twice, bit for bit."""
    page = 64
    made, out, lse = run(lengths, page, heads, BF, "auto", q_lens=q_lens, seed=3)
    q, k, v, table, scale = made
    see = S.see_paged(table, lengths, page, q_lens)
    pick = sorted(set(range(0, sum(q_lens), 211)) | {sum(q_lens) - 1} | {c for c in A.cu(q_lens) if c < sum(q_lens)})
    A.check(out[pick], lse[pick], S.attend(q[pick], k.flatten(0, 1), v.flatten(0, 1), [see[r] for r in pick], scale))
    assert torch.isfinite(out).all()
    _, again, alse = run(lengths, page, heads, BF, "auto", q_lens=q_lens, tensors=made[:3], pool=(None, table))
    assert torch.equal(out, again) and torch.equal(lse, alse)


def test_long_sequences_with_bad_lengths_and_pages():
    """Long enough without the bad one that the call still takes whole row tiles by its lengths."""
    heads, page, n, lengths = (128, 1, 64), 64, 1030, [14000, 14000, 14000]
    q_lens, rows = [n] * 3, 3 * n
    total, table = S.pool(lengths, page, random.Random(5))
    q, k, v = make(5, rows, total, page, heads, BF)
    ws = K.new_attention_workspace(rows, 3, *heads, BF)
    see = S.see_paged(table, lengths, page, q_lens)
    pick = list(range(0, n, 97)) + list(range(2 * n, rows, 97))
    ref = S.attend(q[pick], k.flatten(0, 1), v.flatten(0, 1), [see[r] for r in pick], 0.09)
    for what in ("length", "page"):
        held, t = list(lengths), table.clone()
        if what == "length":
            held[1] = 2 ** 31 - 1
        else:
            t[1, 3] = total
        out = torch.full_like(q, math.nan)
        out, lse = K.kpool_attention_paged(q, k, v, t.cuda(), i32(held), 0.09, cu_q=i32(A.cu(q_lens)), out=out, return_lse=True,
                                           workspace=ws)
        assert K.kpool_last_device_error(ws) == K.KPOOL_ERR_INVALID_ARG
        A.check(out[pick], lse[pick], ref, what)
        if what == "length":
            assert (out[n:2 * n] == 0).all() and (lse[n:2 * n] == -math.inf).all()
