"""Attention over short lists of selected tokens on the GPU: a warp per item, by the rule on sizes,
against the plain 64-bit implementation at widths around its steps of 16 ids, one and two halves of 8 heads, few
rows (an item shared by four warps) and many (one each); and the same checks as other selections
with the tcgen05 kernels asked for, which short lists no longer reach by themselves."""
import functools
import math

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A
from tests import test_gpu_attention as G
from tests.test_gpu_attention import BF, i32, make, strided

pytestmark = pytest.mark.gpu
HEADS = [(4, 4, 128), (8, 2, 64), (8, 1, 128), (9, 1, 64), (24, 2, 128), (16, 1, 64), (34, 2, 64), (64, 1, 128)]


def lists(seed, rows, lens, width):
    """Random ids, some empty, some named twice, some outside; rows without any, rows of one."""
    g = torch.Generator().manual_seed(seed)
    seq = [b for b in range(len(lens)) if lens[b]]
    seq = [seq[i % len(seq)] for i in range(rows)]
    top = torch.tensor([lens[b] for b in seq])
    ids = (torch.rand((rows, width), generator=g) * top[:, None]).to(torch.int32)
    ids[torch.rand(ids.shape, generator=g) < 0.15] = -1
    if width:
        ids[1::7, 0] = 2 ** 31 - 1
        ids[2::7, -1] = -2 ** 31
        ids[3::7] = -1
        ids[4::7, 1:] = -1
        ids[5::7, -1] = ids[5::7, 0]
    return ids, seq


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("rows", [1, 23, 700])
@pytest.mark.parametrize("width", [0, 1, 15, 16, 17, 33, 68])
def test_short_lists(width, rows, heads):
    lens = [90, 0, 1, 230]
    ids, seq = lists(width + rows, rows, lens, width)
    q, k, v = make(width, rows, sum(lens), heads, BF)
    scale = 1.0 / math.sqrt(heads[2])
    ws = K.new_attention_workspace(rows, len(lens), *heads, BF)
    out, lse = K.kpool_attention_selected(q, k, v, ids.cuda(), i32(A.cu(lens)), scale, row_seq=i32(seq),
                                          return_lse=True, workspace=ws)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    A.check(out, lse, A.reference(q, k, v, A.see_selected(ids, seq, lens), scale))
    again, lse2 = K.kpool_attention_selected(q, k, v, ids.cuda(), i32(A.cu(lens)), scale, row_seq=i32(seq),
                                             return_lse=True, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 1, 64)], ids=str)
@pytest.mark.parametrize("how", ["heads_first", "beside", "stacked"])
def test_strides_of_short_lists(how, heads):
    lens, rows = [70, 121], 50
    ids, seq = lists(3, rows, lens, 20)
    q, k, v = make(12, rows, 191, heads, BF)
    guard = torch.full((rows, heads[0] + 2, heads[2] + 16), 7.0, dtype=BF, device="cuda")
    out = guard[:, 1:-1, 8:8 + heads[2]]
    _, lse = K.kpool_attention_selected(*[strided(t, how) for t in (q, k, v)], ids.cuda(), i32(A.cu(lens)), 0.09,
                                        row_seq=i32(seq), out=out, return_lse=True)
    A.check(out, lse, A.reference(q, k, v, A.see_selected(ids, seq, lens), 0.09))
    out.fill_(7.0)
    assert (guard == 7.0).all()


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("width", [20, 60])
def test_unnamed_tokens_do_not_matter_and_named_ones_show(width, bad):
    heads, rows, n = (12, 1, 128), 30, 200
    ids, seq = lists(width, rows, [n], width)
    ids[ids >= 0] //= 2
    ids[ids == 50] = 51
    q, k, v = make(15, rows, n, heads, BF)
    see = A.see_selected(ids, seq, [n])
    ref = A.reference(q, k, v, see, 0.1)
    for t in (k, v):
        t[100:] = bad
        t[50] = bad
    args = (q, k, v, ids.cuda(), i32([0, n]), 0.1)
    out, lse = K.kpool_attention_selected(*args, row_seq=i32(seq), return_lse=True)
    A.check(out, lse, ref)
    k[0] = v[0] = 0
    v[0, 0, 5] = bad
    out = K.kpool_attention_selected(*args, row_seq=i32(seq))[0].cpu()
    has = torch.tensor([bool((j == 0).any()) for j in see])
    assert 0 < has.sum() < rows
    assert torch.isfinite(out[~has]).all()
    want = torch.full_like(out[has][:, :, 5], bad)
    assert torch.equal(torch.isnan(out[has][:, :, 5]), torch.isnan(want))
    assert math.isnan(bad) or torch.equal(out[has][:, :, 5], want)
    out[:, :, 5] = 0
    assert torch.isfinite(out).all()


def test_scores_of_minus_infinity_give_no_weight():
    q = torch.ones((3, 2, 64), dtype=BF, device="cuda")
    k = torch.zeros((3, 2, 64), dtype=BF, device="cuda")
    v = torch.randn((3, 2, 64), device="cuda").to(BF)
    k[0, :, 0] = -float("inf")
    ids = i32([[0, -1], [0, 1], [2, 1]])
    out, lse = K.kpool_attention_selected(q, k, v, ids, i32([0, 3]), 1.0, row_seq=i32([0] * 3), return_lse=True)
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()
    ref = A.reference(q[1:], torch.zeros_like(k), v, [torch.tensor([1]), torch.tensor([1, 2])], 1.0)
    A.check(out[1:], lse[1:], ref)


@pytest.mark.parametrize("width", [20, 68])
def test_short_lists_on_streams_and_in_graphs(width):
    heads = (8, 2, 128)
    ids, seq = lists(5, 40, [300], width)
    q, k, v = make(18, 40, 300, heads, BF)
    ws = K.new_attention_workspace(40, 1, *heads, BF)
    out, lse, dev, rs, ck = torch.empty_like(q), torch.empty((40, 8), device="cuda"), ids.cuda(), i32(seq), i32([0, 300])

    def call(stream=None):
        K.kpool_attention_selected(q, k, v, dev, ck, 0.1, row_seq=rs, out=out, out_lse=lse, workspace=ws, stream=stream)
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
    out.zero_()
    ws.fill_(0xA5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK


@pytest.fixture
def tcgen05(monkeypatch):
    """Selections on the tcgen05 kernels whatever their lists."""
    call = K.kpool_attention_selected
    monkeypatch.setattr(K, "kpool_attention_selected", lambda *a, **kw: call(*a, **{**kw, "score_kernel": K.KPOOL_SCORE_TC}))


SMALL = [h for h in G.SELECT_HEADS if h[3] == BF and h[2] in (64, 128)]


@pytest.mark.parametrize("heads", SMALL, ids=str)
@pytest.mark.parametrize("width", [1, 20, 131])
def test_selected_on_tcgen05(width, heads, tcgen05):
    G.test_selected(width, heads, "auto")


@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 1, 64), (40, 1, 128)], ids=str)
@pytest.mark.parametrize("rows", [1, 40, 700])
def test_few_and_many_rows_on_tcgen05(rows, heads, tcgen05):
    G.test_selected_few_and_many_rows(rows, heads, "auto")


@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 1, 64), (12, 2, 128)], ids=str)
@pytest.mark.parametrize("kind", ["causal", "any", "twice", "bad_ids"])
def test_whole_prompt_on_tcgen05(kind, heads, tcgen05):
    G.test_selected_whole_prompt(kind, heads)


@pytest.mark.parametrize("bad", G.BAD)
@pytest.mark.parametrize("heads", [(8, 2, 128, BF), (4, 4, 64, BF)], ids=str)
def test_unseen_on_tcgen05(heads, bad, tcgen05):
    G.test_unseen_keys_and_values_do_not_matter(heads, bad, "auto")


@pytest.mark.parametrize("check", ["every", "no_keys", "graphs", "errors"])
def test_others_on_tcgen05(check, tcgen05):
    {"every": G.test_selected_every_token_is_prompt, "no_keys": G.test_no_keys_at_all,
     "graphs": functools.partial(G.test_streams_and_graphs_repeat_bit_for_bit, "selected"),
     "errors": G.test_device_errors_are_reported}[check]()
