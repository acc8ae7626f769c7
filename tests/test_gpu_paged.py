"""Attention over a cache in pages on the GPU against a plain 64-bit implementation, through the public entry
point, on both kernel families."""
import math
import random

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A
from tests import serving_reference as S

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FAMILIES = {"auto": K.KPOOL_SCORE_AUTO, "simt": K.KPOOL_SCORE_SIMT}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(seed, rows, pages, page, heads, dtype):
    hq, hkv, d = heads
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((rows, hq, d), generator=g) * 2).to(dtype).cuda()
    k = torch.randn((pages, page, hkv, d), generator=g).to(dtype).cuda()
    v = torch.randn((pages, page, hkv, d), generator=g).to(dtype).cuda()
    return q, k, v


def run(lengths, page, heads, dtype, family, q_lens=None, seed=1, tensors=None, pool=None, poison=True):
    rows = sum(q_lens) if q_lens else len(lengths)
    total, table = pool or S.pool(lengths, page, random.Random(seed))
    q, k, v = tensors or make(seed, rows, total, page, heads, dtype)
    scale = 1.0 / math.sqrt(heads[2])
    ws = K.new_attention_workspace(rows, len(lengths), *heads, dtype)
    kw = {}
    if poison:  # a place that is never written shows
        ws.fill_(0xFF)
        kw = dict(out=torch.full_like(q, math.nan), out_lse=torch.full(q.shape[:2], math.nan, device="cuda"))
    out, lse = K.kpool_attention_paged(q, k, v, table.cuda(), i32(lengths), scale,
                                       cu_q=i32(A.cu(q_lens)) if q_lens else None, return_lse=True, workspace=ws,
                                       score_kernel=FAMILIES[family], **kw)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    return (q, k, v, table, scale), out, lse


def verify(made, out, lse, lengths, page, q_lens=None, what=""):
    q, k, v, table, scale = made
    see = S.see_paged(table, lengths, page, q_lens or [1] * len(lengths))
    A.check(out, lse, S.attend(q, k.flatten(0, 1), v.flatten(0, 1), see, scale), what)


HEADS = [(8, 2, 128, BF), (16, 1, 64, BF), (6, 2, 128, BF), (4, 4, 64, F32), (6, 2, 96, F32), (4, 2, 256, BF), (3, 1, 24, BF)]


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 100, 128, 200, 256])
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_decode(heads, page, family):
    lengths = [1, 130, 0, 257, 64, 15, 1000]
    verify(*run(lengths, page, heads[:3], heads[3], family, seed=page), lengths, page)


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("page", [1, 16, 20, 128])
@pytest.mark.parametrize("heads", [(8, 2, 128, BF), (16, 1, 64, BF), (4, 4, 32, F32)], ids=str)
def test_chunks(heads, page, family):
    """The newest rows of every sequence: whole prompts, chunks, single tokens, none, more rows than keys."""
    q_lens, lengths = [70, 0, 1, 40, 9, 129], [70, 33, 200, 300, 4, 500]
    verify(*run(lengths, page, heads[:3], heads[3], family, q_lens=q_lens, seed=page), lengths, page, q_lens)


@pytest.mark.parametrize("heads,lengths,page", [
    ((32, 8, 128), [5000, 37, 9001, 12288], 16), ((64, 1, 128), [20000], 64), ((16, 1, 64), [30000, 1], 8),
    ((8, 8, 128), [700] * 30, 128), ((32, 8, 128), [1] * 200, 16), ((24, 4, 64), [3000] * 12, 48)], ids=str)
def test_long_caches(heads, lengths, page):
    """Rows cut over CTAs and joined; the same call twice, bit for bit."""
    made, out, lse = run(lengths, page, heads, BF, "auto", seed=5)
    verify(made, out, lse, lengths, page)
    _, again, alse = run(lengths, page, heads, BF, "auto", seed=5, tensors=made[:3], pool=(None, made[3]))
    assert torch.equal(out, again) and torch.equal(lse, alse)


@pytest.mark.parametrize("heads", [(128, 1, 64), (80, 2, 128), (20, 1, 64), (24, 2, 128), (7, 7, 128)], ids=str)
@pytest.mark.parametrize("page", [16, 64])
def test_group_sizes(page, heads):
    lengths = [300, 1, 129, 0, 2000]
    verify(*run(lengths, page, heads, BF, "auto", seed=page), lengths, page)


@pytest.mark.parametrize("page", [1, 16, 128])
def test_decode_as_chunks_of_one_row(page):
    """cu_q that gives every sequence one row: another form of the kernel, the same rows."""
    lengths, heads = [700, 3, 0, 4000], (8, 2, 128)
    verify(*run(lengths, page, heads, BF, "auto", q_lens=[1] * 4, seed=page), lengths, page, [1] * 4)


@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 1, 64)], ids=str)
def test_drafted_rows(heads):
    """A few rows a sequence, as drafts are verified, over long and short caches."""
    q_lens, lengths = [4, 5, 1, 8, 3], [9000, 64, 1, 130, 3]
    verify(*run(lengths, 16, heads, BF, "auto", q_lens=q_lens, seed=31), lengths, 16, q_lens)


SMALL_PAGES = [1, 2, 3, 6, 130]  # pieces of one or two tokens


@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 1, 64), (6, 2, 128), (128, 1, 128)], ids=str)
@pytest.mark.parametrize("page", SMALL_PAGES)
def test_chunks_over_small_pages(page, heads):
    """Many tiles a run, sequences of one to all of their rows; the same call twice, bit for bit."""
    q_lens, lengths = [300, 1, 0, 7, 129, 64], [3001, 127, 50, 129, 129, 2048]
    made, out, lse = run(lengths, page, heads, BF, "auto", q_lens=q_lens, seed=page)
    verify(made, out, lse, lengths, page, q_lens)
    _, again, alse = run(lengths, page, heads, BF, "auto", q_lens=q_lens, tensors=made[:3], pool=(None, made[3]))
    assert torch.equal(out, again) and torch.equal(lse, alse)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("page", SMALL_PAGES)
def test_behind_the_last_key_of_small_pages(page, bad):
    lengths, heads, q_lens = [150, 20, 700, 0, 128], (8, 2, 128), [3, 1, 40, 1, 128]
    total, table = S.pool(lengths, page, random.Random(40))
    q, k, v = make(40, sum(q_lens), total, page, heads, BF)
    free = torch.ones(total * page, dtype=torch.bool, device="cuda")
    free[torch.cat(S.slots(table, lengths, page)).cuda()] = False
    kb, vb = k.clone(), v.clone()
    for t in (kb, vb):
        t.flatten(0, 1)[free] = bad
    made, out, lse = run(lengths, page, heads, BF, "auto", q_lens=q_lens, tensors=(q, kb, vb), pool=(total, table))
    verify((q, k, v, table, made[4]), out, lse, lengths, page, q_lens)


def test_seen_nan_and_infinite_values_in_small_pages():
    page, lengths, q_lens = 2, [200], [150]
    total, table = S.pool(lengths, page, random.Random(41))
    q, k, v = make(41, 150, total, page, (4, 2, 128), BF)
    at = S.slots(table, lengths, page)[0]
    v.flatten(0, 1)[at[130], 0, 5] = math.nan
    v.flatten(0, 1)[at[140], 1, 7] = math.inf
    _, out, _ = run(lengths, page, (4, 2, 128), BF, "auto", q_lens=q_lens, tensors=(q, k, v), pool=(total, table))
    nan, inf = torch.isnan(out), torch.isinf(out)
    assert nan[80:, :2, 5].all() and not nan[:80].any() and nan.sum() == 70 * 2
    assert (out[90:, 2:, 7] == math.inf).all() and inf.sum() == 60 * 2


def test_small_pages_apart_and_not_there():
    """Pages with a gap between them (another form), and one that the pool does not have, reported."""
    lengths, heads, q_lens, page = [300, 40], (8, 2, 128), [90, 40], 2
    total, table = S.pool(lengths, page, random.Random(42))
    q, k, v = make(42, 130, total, page, heads, BF)
    apart = [torch.full((total, 3, 2, 128), math.nan, dtype=BF, device="cuda")[:, :2] for _ in range(2)]
    for t, x in zip(apart, (k, v)):
        t.copy_(x)
    made, out, lse = run(lengths, page, heads, BF, "auto", q_lens=q_lens, tensors=(q, *apart), pool=(total, table))
    verify((q, k, v, table, made[4]), out, lse, lengths, page, q_lens)
    ws = K.new_attention_workspace(130, 2, *heads, BF)
    for bad in (total, -1, 2 ** 31 - 1):
        t = table.clone()
        t[0, 70] = bad
        got, glse = K.kpool_attention_paged(q, k, v, t.cuda(), i32(lengths), made[4], cu_q=i32([0, 90, 130]),
                                            return_lse=True, workspace=ws)
        assert K.kpool_last_device_error(ws) == K.KPOOL_ERR_INVALID_ARG
        see = S.see_paged(table, lengths, page, q_lens)
        ref = S.attend(q, k.flatten(0, 1), v.flatten(0, 1), see, made[4])
        A.check(got[90:], glse[90:], [x[90:] for x in ref])


def test_more_sequences_than_the_runs_take():
    lengths = [(i * 7) % 40 for i in range(9000)]
    (q, k, v, table, scale), out, lse = run(lengths, 16, (2, 1, 64), BF, "auto", seed=6)
    pick = list(range(0, 9000, 61))
    see = S.see_paged(table, lengths, 16, [1] * 9000)
    ref = S.attend(q[pick], k.flatten(0, 1), v.flatten(0, 1), [see[r] for r in pick], scale)
    A.check(out[pick], lse[pick], ref)


@pytest.mark.parametrize("family", FAMILIES)
def test_same_as_a_contiguous_cache(family):
    """One page per sequence is a cache of slots: the results of the tree operator."""
    lengths, slot, heads = [100, 300, 7], 300, (8, 2, 128)
    q, k, v = make(7, 3, 3, slot, heads, BF)
    (_, _, _, table, scale), out, lse = run(lengths, slot, heads, BF, family, tensors=(q, k, v),
                                            pool=(3, torch.tensor([[2], [0], [1]], dtype=torch.int32)))
    order = [2, 0, 1]
    want, wlse = K.kpool_attention_tree(q, k[order].flatten(0, 1), v[order].flatten(0, 1), i32([0, 1, 2, 3]),
                                        i32([0, 300, 600, 900]), i32([n - 1 for n in lengths]), scale, return_lse=True,
                                        score_kernel=FAMILIES[family])
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("family", FAMILIES)
def test_shared_pages(family):
    """Two sequences with the same first pages, and a page that appears twice in one table."""
    page, heads, lengths = 16, (8, 2, 128), [40, 45, 60]
    table = torch.tensor([[3, 1, 4, 0], [3, 1, 5, 0], [2, 2, 6, 2]], dtype=torch.int32)
    tensors = make(8, 3, 7, page, heads, BF)
    verify(*run(lengths, page, heads, BF, family, tensors=tensors, pool=(7, table)), lengths, page)


@pytest.mark.parametrize("how", ["heads_first", "beside", "pages_apart"])
@pytest.mark.parametrize("heads", [(8, 2, 128, BF), (4, 4, 32, F32)], ids=str)
def test_strides(heads, how):
    lengths, page = [50, 1, 140], 16
    total, table = S.pool(lengths, page, random.Random(9))
    q, k, v = make(9, 3, total, page, heads[:3], heads[3])

    def strided(t):
        n, size, h, d = t.shape
        if how == "heads_first":
            return t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        if how == "beside":
            big = torch.full((n, size, h, 2 * d + 8), math.nan, dtype=t.dtype, device="cuda")
            big[..., d:2 * d] = t
            return big[..., d:2 * d]
        big = torch.full((n, 3, size + 1, h + 1, d), math.nan, dtype=t.dtype, device="cuda")
        big[:, 1, :size, :h] = t
        return big[:, 1, :size, :h]
    made, out, lse = run(lengths, page, heads[:3], heads[3], "auto", tensors=(q, strided(k), strided(v)), pool=(total, table))
    verify((q, k, v, table, made[4]), out, lse, lengths, page)


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_what_lies_behind_the_last_key_does_not_matter(page, bad, family):
    lengths, heads, q_lens = [150, 20, 300, 0], (8, 2, 128), [3, 1, 40, 1]
    total, table = S.pool(lengths, page, random.Random(10))
    q, k, v = make(10, 45, total, page, heads, BF)
    used = torch.cat(S.slots(table, lengths, page)).cuda()
    free = torch.ones(total * page, dtype=torch.bool, device="cuda")
    free[used] = False
    kb, vb = k.clone(), v.clone()
    for t in (kb, vb):
        t.flatten(0, 1)[free] = bad
    made, out, lse = run(lengths, page, heads, BF, family, q_lens=q_lens, tensors=(q, kb, vb), pool=(total, table))
    verify((q, k, v, table, made[4]), out, lse, lengths, page, q_lens)


@pytest.mark.parametrize("family", FAMILIES)
def test_seen_nan_and_infinite_values_show(family):
    page, lengths, q_lens = 16, [200], [150]
    total, table = S.pool(lengths, page, random.Random(11))
    q, k, v = make(11, 150, total, page, (4, 2, 128), BF)
    at = S.slots(table, lengths, page)[0]
    v.flatten(0, 1)[at[130], 0, 5] = math.nan
    v.flatten(0, 1)[at[140], 1, 7] = math.inf
    _, out, _ = run(lengths, page, (4, 2, 128), BF, family, q_lens=q_lens, tensors=(q, k, v), pool=(total, table))
    nan, inf = torch.isnan(out), torch.isinf(out)
    first = 130 - 50
    assert nan[first:, :2, 5].all() and not nan[:first].any() and nan.sum() == 70 * 2
    assert (out[90:, 2:, 7] == math.inf).all() and inf.sum() == 60 * 2


@pytest.mark.parametrize("family", FAMILIES)
def test_offsets_past_32_bits(family):
    """The last pages of a pool of more than 2^32 bytes; what lies before them is not set."""
    pages, page, heads = 36000, 64, (16, 8, 128)
    k = torch.empty((pages, page, 8, 128), dtype=BF, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() * 2 > 2 ** 32
    q, k[-9:], v[-9:] = make(12, 2, 9, page, heads, BF)
    table = torch.tensor([[pages - 1, pages - 3, pages - 5], [pages - 2, pages - 4, pages - 9]], dtype=torch.int32)
    lengths = [130, 190]
    out, lse = K.kpool_attention_paged(q, k, v, table.cuda(), i32(lengths), 0.1, return_lse=True,
                                       score_kernel=FAMILIES[family])
    see = S.see_paged(table - (pages - 9), lengths, page, [1, 1])
    A.check(out, lse, S.attend(q, k[-9:].flatten(0, 1), v[-9:].flatten(0, 1), see, 0.1))


def test_nothing_to_see():
    q, k, v = make(13, 3, 4, 16, (4, 2, 128), BF)
    for table, keys in ((torch.zeros((3, 0), dtype=torch.int32), k), (torch.zeros((3, 2), dtype=torch.int32), k[:0])):
        out, lse = K.kpool_attention_paged(q, keys, keys, table.cuda(), i32([0, 0, 0]), 0.1, return_lse=True)
        assert (out == 0).all() and (lse == -math.inf).all()
    out, _ = K.kpool_attention_paged(q[:0], k, v, torch.zeros((0, 2), dtype=torch.int32, device="cuda"), i32([]), 0.1)
    assert out.shape == (0, 4, 128)


@pytest.mark.parametrize("family", FAMILIES)
def test_device_errors(family):
    page, heads = 16, (8, 2, 128)
    q, k, v = make(14, 3, 6, page, heads, BF)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32)
    ws = K.new_attention_workspace(3, 3, *heads, BF)
    kw = dict(return_lse=True, workspace=ws, score_kernel=FAMILIES[family])
    ref = S.attend(q, k.flatten(0, 1), v.flatten(0, 1), S.see_paged(table, [20, 30, 25], page, [1] * 3), 0.1)
    for n in (33, -1, 2 ** 31 - 1):  # a length that the table does not hold: that sequence's row is empty
        out, lse = K.kpool_attention_paged(q, k, v, table.cuda(), i32([20, n, 25]), 0.1, **kw)
        assert K.kpool_last_device_error(ws) == K.KPOOL_ERR_INVALID_ARG
        assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
        A.check(out[[0, 2]], lse[[0, 2]], [t[[0, 2]] for t in ref])
    for bad in (6, -1, 2 ** 31 - 1):  # a page outside the pool: reported, the other rows are right
        t = table.clone()
        t[1, 1] = bad
        out, lse = K.kpool_attention_paged(q, k, v, t.cuda(), i32([20, 30, 25]), 0.1, **kw)
        assert K.kpool_last_device_error(ws) == K.KPOOL_ERR_INVALID_ARG
        A.check(out[[0, 2]], lse[[0, 2]], [t[[0, 2]] for t in ref])
    out, lse = K.kpool_attention_paged(q, k, v, table.cuda(), i32([20, 30, 25]), 0.1, cu_q=i32([0, 2, 1, 3]), **kw)
    assert K.kpool_last_device_error(ws) == K.KPOOL_ERR_INVALID_ARG
    out, lse = K.kpool_attention_paged(q, k, v, table.cuda(), i32([20, 30, 25]), 0.1, **kw)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    A.check(out, lse, ref)


def test_streams_graphs_and_growing_caches():
    """A captured step replayed while lengths and tables grow, on a clobbered workspace."""
    page, heads, lengths = 16, (8, 2, 128), [4000, 31, 900]
    total, table = S.pool([n + 64 for n in lengths], page, random.Random(15))
    q, k, v = make(15, 3, total, page, heads, BF)
    ws = K.new_attention_workspace(3, 3, *heads, BF)
    n, t = i32(lengths), table.cuda()
    out, lse = torch.empty_like(q), torch.empty((3, 8), device="cuda")

    def call(stream=None):
        K.kpool_attention_paged(q, k, v, t, n, 0.1, out=out, out_lse=lse, workspace=ws, stream=stream)
    call()
    torch.cuda.synchronize()
    want, wlse = out.clone(), lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    call(side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for step in range(4):
        out.fill_(math.nan)
        ws.fill_(0xA5)
        g.replay()
        torch.cuda.synchronize()
        now = [x + 17 * step for x in lengths]
        see = S.see_paged(table, now, page, [1] * 3)
        A.check(out, lse, S.attend(q, k.flatten(0, 1), v.flatten(0, 1), see, 0.1), f"step {step}")
        n.add_(17)
