"""The attention operators on the GPU against a plain 64-bit implementation, through the
public entry points, on every kernel family: lengths of zero and one, ragged packs, tiles
that end inside a sequence, masks that leave rows empty, strided heads, infinities and NaN
in keys and values that a row does not see, other streams, graphs and device errors."""
import math
import random

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FAMILIES = {"auto": K.KPOOL_SCORE_AUTO, "simt": K.KPOOL_SCORE_SIMT}


def make(seed, rows, tokens, heads, dtype, spread=2.0):
    hq, hkv, d = heads
    g = torch.Generator(device="cpu").manual_seed(seed)
    q = (torch.randn((rows, hq, d), generator=g) * spread).to(dtype).cuda()
    k = torch.randn((tokens, hkv, d), generator=g).to(dtype).cuda()
    v = torch.randn((tokens, hkv, d), generator=g).to(dtype).cuda()
    return q, k, v


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_prompt(ql, kl, heads, dtype, family, seed=1, scale=None, tensors=None, **kw):
    q, k, v = tensors or make(seed, sum(ql), sum(kl), heads, dtype)
    scale = scale or 1.0 / math.sqrt(heads[2])
    ws = K.new_attention_workspace(q.shape[0], len(ql), *heads, dtype)
    out, lse = K.kpool_attention_prompt(q, k, v, i32(A.cu(ql)), i32(A.cu(kl)), scale, return_lse=True, workspace=ws,
                                        score_kernel=FAMILIES[family], **kw)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    return (q, k, v, scale), out, lse


def run_tree(nodes, prefixes, extents, bits, heads, dtype, family, seed=2, tensors=None, words=None):
    q, k, v = tensors or make(seed, sum(nodes), sum(extents), heads, dtype)
    scale = 1.0 / math.sqrt(heads[2])
    mask = None
    if bits:
        words = words or max(1, (max(nodes) + 31) // 32)
        mask = A.mask_words([x for b in bits for x in b], words).cuda()
    ws = K.new_attention_workspace(q.shape[0], len(nodes), *heads, dtype)
    out, lse = K.kpool_attention_tree(q, k, v, i32(A.cu(nodes)), i32(A.cu(extents)), i32(prefixes), scale, mask=mask,
                                      return_lse=True, workspace=ws, score_kernel=FAMILIES[family])
    return (q, k, v, scale), out, lse, ws


HEADS = [(8, 2, 128, BF), (4, 4, 64, BF), (6, 2, 128, BF), (16, 1, 64, BF), (8, 8, 64, F32), (4, 4, 32, F32),
         (6, 2, 96, F32), (4, 2, 256, F32), (3, 1, 24, BF)]
PACKS = [
    ([1], [1]),
    ([0, 5, 0, 1, 33], [0, 5, 0, 1, 33]),
    ([127, 128, 129], [127, 128, 129]),
    ([31, 1, 257], [300, 700, 257]),
    ([9, 40], [4, 0]),             # fewer keys than rows: the first rows see nothing
]


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("pack", range(len(PACKS)))
def test_prompt(pack, heads, family):
    ql, kl = PACKS[pack]
    (q, k, v, scale), out, lse = run_prompt(ql, kl, heads[:3], heads[3], family, seed=10 + pack)
    A.check(out, lse, A.reference(q, k, v, A.see_prompt(ql, kl), scale))


@pytest.mark.parametrize("heads", [(4, 1, 128, BF), (2, 2, 64, BF), (128, 1, 64, BF), (80, 2, 128, BF), (2, 1, 64, F32)],
                         ids=str)
def test_prompt_longer(heads):
    ql, kl = [70, 500, 3], [900, 500, 1500]
    (q, k, v, scale), out, lse = run_prompt(ql, kl, heads[:3], heads[3], "auto", seed=31)
    A.check(out, lse, A.reference(q, k, v, A.see_prompt(ql, kl), scale))


@pytest.mark.parametrize("scale", [1e-4, 1.0, 6.0])
def test_prompt_scales(scale):
    """Nearly uniform weights, and weights that are all but one zero (large running maxima)."""
    ql = [300]
    (q, k, v, _), out, lse = run_prompt(ql, ql, (4, 2, 128), BF, "auto", seed=5, scale=scale)
    A.check(out, lse, A.reference(q, k, v, A.see_prompt(ql, ql), scale))


def test_prompt_rising_scores():
    """Scores that grow along the keys move the running maximum at every tile."""
    n = 600
    q, k, v = make(6, n, n, (2, 1, 64), BF)
    q = q.abs()
    k = (k.abs() * (1 + torch.arange(n, device="cuda") / 40)[:, None, None]).to(BF)
    (q, k, v, scale), out, lse = run_prompt([n], [n], (2, 1, 64), BF, "auto", tensors=(q, k, v))
    A.check(out, lse, A.reference(q, k, v, A.see_prompt([n], [n]), scale))


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("chain", [True, False])
def test_tree(chain, heads, family):
    rng = random.Random(3)
    nodes, prefixes, extents = [1, 7, 0, 40, 5], [130, 0, 9, 300, 1000], [256, 7, 40, 345, 1024]
    bits = None if chain else [A.random_tree(n, rng) for n in nodes]
    (q, k, v, scale), out, lse, ws = run_tree(nodes, prefixes, extents, bits, heads[:3], heads[3], family)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    A.check(out, lse, A.reference(q, k, v, A.see_tree(nodes, extents, prefixes, bits), scale))


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("heads", [(8, 2, 128, BF), (4, 4, 64, F32)], ids=str)
def test_tree_wide(heads, family):
    """More nodes than a tile of keys, more words than nodes need, bits beyond the nodes set."""
    rng = random.Random(4)
    nodes, prefixes, extents = [200, 65], [77, 640], [300, 800]
    bits = [[x | (1 << 250) | (1 << 287) for x in A.random_tree(n, rng)] for n in nodes]
    (q, k, v, scale), out, lse, ws = run_tree(nodes, prefixes, extents, bits, heads[:3], heads[3], family, words=9)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    A.check(out, lse, A.reference(q, k, v, A.see_tree(nodes, extents, prefixes, bits), scale))


@pytest.mark.parametrize("family", FAMILIES)
def test_tree_few_words(family):
    """Nodes beyond the mask's words are seen by no row, themselves included."""
    rng = random.Random(5)
    nodes, prefixes, extents = [50], [70], [130]
    bits = [A.random_tree(50, rng)]
    (q, k, v, scale), out, lse, _ = run_tree(nodes, prefixes, extents, bits, (4, 1, 64), BF, family, words=1)
    cut = [[x & 0xFFFFFFFF for x in bits[0]]]
    A.check(out, lse, A.reference(q, k, v, A.see_tree(nodes, extents, prefixes, cut), scale))


@pytest.mark.parametrize("family", FAMILIES)
def test_tree_rows_that_see_nothing(family):
    nodes, prefixes, extents = [4, 3], [0, 0], [16, 3]
    bits = [[0, 1, 0, 0b1101], [0, 0, 0]]
    (q, k, v, scale), out, lse, _ = run_tree(nodes, prefixes, extents, bits, (4, 1, 128), BF, family)
    A.check(out, lse, A.reference(q, k, v, A.see_tree(nodes, extents, prefixes, bits), scale))
    assert (out[0] == 0).all() and torch.isinf(lse[0]).all()


@pytest.mark.parametrize("heads,nodes,prefixes", [
    ((64, 1, 128), [1, 1], [20000, 3000]), ((16, 1, 64), [40, 3], [8000, 200]), ((8, 8, 128), [1], [30000]),
    ((32, 8, 128), [16, 30, 8], [3000, 1000, 9000]), ((4, 4, 64), [1], [1500]),
], ids=str)
def test_rows_cut_into_many_runs(heads, nodes, prefixes):
    """One item over all CTAs of the GPU: joins of more than a hundred partial results."""
    extents = [p + n for p, n in zip(prefixes, nodes)]
    (q, k, v, scale), out, lse, ws = run_tree(nodes, prefixes, extents, None, heads, BF, "auto", seed=77)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    A.check(out, lse, A.reference(q, k, v, A.see_tree(nodes, extents, prefixes, None), scale))


@pytest.mark.parametrize("heads", [(8, 2, 128, BF), (16, 1, 64, BF), (8, 8, 128, BF)], ids=str)
def test_decode_long_cache(heads):
    """Few rows over long caches: the key axis is split over CTAs and joined."""
    nodes, prefixes = [1, 1, 2, 1], [5000, 37, 9001, 12288]
    extents = [p + n + 11 for p, n in zip(prefixes, nodes)]
    (q, k, v, scale), out, lse, ws = run_tree(nodes, prefixes, extents, None, heads[:3], heads[3], "auto")
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    A.check(out, lse, A.reference(q, k, v, A.see_tree(nodes, extents, prefixes, None), scale))


def test_many_sequences():
    rng = random.Random(8)
    nodes = [rng.choice([0, 1, 1, 2, 3]) for _ in range(300)]
    prefixes = [rng.randrange(0, 200) for _ in nodes]
    extents = [n + p + rng.randrange(3) for n, p in zip(nodes, prefixes)]
    (q, k, v, scale), out, lse, ws = run_tree(nodes, prefixes, extents, None, (4, 2, 64), BF, "auto")
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    A.check(out, lse, A.reference(q, k, v, A.see_tree(nodes, extents, prefixes, None), scale))


@pytest.mark.parametrize("ql,kl,heads", [
    ([500], [500], (128, 1, 128)), ([4000], [4000], (32, 8, 128)), ([70, 500, 3], [900, 500, 1500], (128, 1, 64)),
    ([1] * 40, [3000] * 40, (8, 2, 128)), ([6000, 1, 900], [6000, 7000, 1000], (32, 8, 64)), ([12000], [12000], (32, 8, 128)),
    ([20, 7, 1], [300, 20000, 4000], (24, 4, 64)), ([900, 64, 300], [300, 0, 2000], (8, 2, 128)),
    ([1] * 9 + [1200], [2] * 9 + [1200], (8, 2, 128)), ([1500], [1500], (32, 8, 128)), ([1100], [1100], (8, 8, 128)),
], ids=str)
def test_runs_of_many_segments(ql, kl, heads):
    """Every split of the work (one CTA per row tile; equal runs with several segments, joined or not)
    against the CUDA-core kernel, twice bit for bit."""
    (q, k, v, scale), out, lse = run_prompt(ql, kl, heads, BF, "auto", seed=41)
    _, want, wlse = run_prompt(ql, kl, heads, BF, "simt", tensors=(q, k, v))
    # both sides are within the weights' and the output's rounding of the true value; |v| sums stay below 4
    assert ((out.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -6).all()
    # (rows without a key are -inf on both sides)
    assert torch.where(wlse == -math.inf, lse == wlse, (lse - wlse).abs() <= 1e-4).all()
    _, again, alse = run_prompt(ql, kl, heads, BF, "auto", tensors=(q, k, v))
    assert torch.equal(out, again) and torch.equal(lse, alse)


@pytest.mark.parametrize("lens", [[1] * 9000, [1] * 8900 + [60, 0, 200]], ids=["ones", "mixed"])
def test_more_sequences_than_the_runs_take(lens):
    heads = (2, 1, 64)
    (q, k, v, scale), out, lse = run_prompt(lens, lens, heads, BF, "auto", seed=91)
    pick = sorted(set(range(0, sum(lens), 97)) | set(range(max(0, sum(lens) - 40), sum(lens))))
    see = A.see_prompt(lens, lens)
    A.check(out[pick], lse[pick], A.reference(q[pick], k, v, [see[r] for r in pick], scale))


@pytest.mark.parametrize("family", FAMILIES)
def test_offsets_past_32_bits(family):
    """The last tokens of a cache of more than 2^32 bytes; what lies before them is not set."""
    tokens, heads = 2_300_000, (16, 8, 128)
    k = torch.empty((tokens, 8, 128), dtype=BF, device="cuda")
    v = torch.empty((tokens, 8, 128), dtype=BF, device="cuda")
    assert k.numel() * 2 > 2 ** 32
    n = 500
    q, k[-n:], v[-n:] = make(92, 6, n, heads, BF)
    lens = [tokens - n, n]
    nodes, prefixes, scale = [0, 6], [0, n - 6], 0.1
    kw = dict(return_lse=True, score_kernel=FAMILIES[family])
    cu = i32(A.cu(lens))
    out, lse = K.kpool_attention_tree(q, k, v, i32(A.cu(nodes)), cu, i32(prefixes), scale, **kw)
    ref = A.reference(q, k[-n:], v[-n:], A.see_tree([6], [n], [n - 6], None), scale)
    A.check(out, lse, ref, "tree")
    out, lse = K.kpool_attention_prompt(q, k, v, i32(A.cu(nodes)), cu, scale, **kw)
    A.check(out, lse, ref, "prompt")
    ids = torch.randint(0, n, (6, 70), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    out, lse = K.kpool_attention_selected(q, k, v, ids.cuda(), cu, scale, row_seq=i32([1] * 6), **kw)
    A.check(out, lse, A.reference(q, k[-n:], v[-n:], A.see_selected(ids, [0] * 6, [n]), scale), "selected")
    one = i32([0, tokens])     # and as ids of one long sequence
    out, lse = K.kpool_attention_selected(q, k, v, (ids + (tokens - n)).cuda(), one, scale, row_seq=i32([0] * 6), **kw)
    A.check(out, lse, A.reference(q, k[-n:], v[-n:], A.see_selected(ids, [0] * 6, [n]), scale), "long ids")


SELECT_HEADS = HEADS + [(32, 8, 128, BF), (64, 1, 128, BF), (20, 1, 64, BF), (24, 2, 128, BF)]


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("heads", SELECT_HEADS, ids=str)
@pytest.mark.parametrize("width", [1, 20, 131])
def test_selected(width, heads, family):
    lens, rows = [90, 0, 300], 9
    g = torch.Generator().manual_seed(width)
    seq = [0, 2, 2, 0, 2, 0, 2, 2, 0]
    ids = torch.stack([torch.randint(0, lens[b], (width,), generator=g) for b in seq]).to(torch.int32)
    ids[torch.rand(ids.shape, generator=g) < 0.2] = -1
    ids[3] = -1                      # a row without any id
    ids[4] = torch.where(torch.arange(width) % 2 == 0, torch.tensor(10 ** 9, dtype=torch.int32), ids[4])
    q, k, v = make(width, rows, sum(lens), heads[:3], heads[3])
    scale = 1.0 / math.sqrt(heads[2])
    ws = K.new_attention_workspace(rows, 3, *heads[:3], heads[3])
    out, lse = K.kpool_attention_selected(q, k, v, ids.cuda(), i32(A.cu(lens)), scale, row_seq=i32(seq),
                                          return_lse=True, workspace=ws, score_kernel=FAMILIES[family])
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    A.check(out, lse, A.reference(q, k, v, A.see_selected(ids, seq, lens), scale))


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 1, 64), (40, 1, 128)], ids=str)
@pytest.mark.parametrize("rows", [1, 40, 700])
def test_selected_few_and_many_rows(rows, heads, family):
    """One row spreads over CTAs by its ids, many rows go one by one."""
    lens, width = [1500], 1030
    g = torch.Generator().manual_seed(rows)
    ids = torch.stack([torch.randperm(lens[0], generator=g)[:width] for _ in range(rows)]).to(torch.int32)
    ids[rows // 2, 17:900] = -1
    q, k, v = make(rows, rows, lens[0], heads, BF)
    ws = K.new_attention_workspace(rows, 1, *heads, BF)
    out, lse = K.kpool_attention_selected(q, k, v, ids.cuda(), i32([0, lens[0]]), 0.1, row_seq=i32([0] * rows),
                                          return_lse=True, workspace=ws, score_kernel=FAMILIES[family])
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    pick = sorted({0, rows // 2, rows - 1, rows // 3, rows // 7})
    ref = A.reference(q[pick], k, v, A.see_selected(ids[pick], [0] * len(pick), lens), 0.1)
    A.check(out[pick], lse[pick], ref)


def test_selected_every_token_is_prompt():
    """Ids that name every earlier token give the causal result; rows find their own sequences."""
    lens, heads = [37, 0, 64], (8, 2, 128)
    q, k, v = make(9, 101, 101, heads, BF)
    pos = torch.cat([torch.arange(n) for n in lens])
    ids = torch.where(torch.arange(64)[None, :] <= pos[:, None], torch.arange(64)[None, :], -1).to(torch.int32).cuda()
    out, lse = K.kpool_attention_selected(q, k, v, ids, i32(A.cu(lens)), 0.1, return_lse=True)
    ref = A.reference(q, k, v, A.see_prompt(lens, lens), 0.1)
    A.check(out, lse, ref)
    out2, lse2 = K.kpool_attention_prompt(q, k, v, i32(A.cu(lens)), i32(A.cu(lens)), 0.1, return_lse=True)
    A.check(out2, lse2, ref)


@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 1, 64), (12, 2, 128)], ids=str)
@pytest.mark.parametrize("kind", ["causal", "any", "twice", "bad_ids"])
def test_selected_whole_prompt(kind, heads):
    """A packed prompt whose rows attend to selected tokens (also as masked dense attention): ids in
    rank order, ids after the row's own token, ids named twice, ids outside the sequence."""
    lens = [700, 0, 1, 333, 129]
    T, width = sum(lens), 150
    g = torch.Generator().manual_seed(len(kind))
    ids = torch.full((T, width), -1, dtype=torch.int32)
    seq, pos = [], []
    for b, n in enumerate(lens):
        seq += [b] * n
        pos += list(range(n))
    for r in range(T):
        top = lens[seq[r]] if kind == "any" else pos[r] + 1
        pick = torch.randperm(top, generator=g)[:width - 9].to(torch.int32)
        ids[r, :pick.numel()] = pick
    if kind == "twice":
        ids[5:T:17, -1] = ids[5:T:17, 0]
        ids[40:T:50, 3] = ids[40:T:50, 2]
    if kind == "bad_ids":
        ids[::3, 4] = 10 ** 6
        ids[::5, 6] = -7
        ids[9] = -1
    q, k, v = make(21, T, T, heads, BF)
    ws = K.new_attention_workspace(T, len(lens), *heads, BF)
    out, lse = K.kpool_attention_selected(q, k, v, ids.cuda(), i32(A.cu(lens)), 0.1, return_lse=True, workspace=ws)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    A.check(out, lse, A.reference(q, k, v, A.see_selected(ids, seq, lens), 0.1))
    # tokens nobody named may hold anything
    named = torch.zeros(T, dtype=torch.bool)
    for j in A.see_selected(ids[:200], seq[:200], lens):
        named[j] = True
    ids[200:] = -1
    kb, vb = k.clone(), v.clone()
    for t in (kb, vb):
        t[(~named).cuda()] = float("nan")
    out, lse = K.kpool_attention_selected(q, kb, vb, ids.cuda(), i32(A.cu(lens)), 0.1, return_lse=True, workspace=ws)
    A.check(out, lse, A.reference(q, k, v, A.see_selected(ids, seq, lens), 0.1), "unnamed")


def strided(t, how):
    n, h, d = t.shape
    if how == "heads_first":            # [H, T, D]
        return t.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    if how == "beside":                 # beside another tensor in one row
        big = torch.full((n, h, 2 * d + 8), float("nan"), dtype=t.dtype, device="cuda")
        big[:, :, d:2 * d] = t
        return big[:, :, d:2 * d]
    big = torch.full((n, 3, h + 1, d), float("nan"), dtype=t.dtype, device="cuda")   # one of three stacked tensors
    big[:, 1, :h] = t
    return big[:, 1, :h]


@pytest.mark.parametrize("heads", [(8, 2, 128, BF), (4, 4, 64, BF), (4, 2, 32, F32)], ids=str)
@pytest.mark.parametrize("how", ["heads_first", "beside", "stacked"])
def test_strides(how, heads):
    ql, dt = [50, 1, 140], heads[3]
    q, k, v = make(12, 191, 191, heads[:3], dt)
    st = [strided(t, how) for t in (q, k, v)]
    guard = torch.full((191, heads[0] + 2, heads[2] + 16), 7.0, dtype=dt, device="cuda")
    out = guard[:, 1:-1, 8:8 + heads[2]]
    scale = 0.09
    c = i32(A.cu(ql))
    _, lse = K.kpool_attention_prompt(*st, c, c, scale, out=out, return_lse=True)
    A.check(out, lse, A.reference(q, k, v, A.see_prompt(ql, ql), scale))
    keep = guard.clone()
    keep[:, 1:-1, 8:8 + heads[2]] = 7.0
    assert (keep == 7.0).all(), "wrote outside the output's heads"
    ids = torch.randint(0, 140, (191, 33), dtype=torch.int32, device="cuda")
    out.fill_(0)
    _, lse = K.kpool_attention_selected(*st, ids, c, scale, row_seq=i32([2] * 191), out=out, return_lse=True)
    A.check(out, lse, A.reference(q, k, v, A.see_selected(ids, [2] * 191, ql), scale))


BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("heads", [(8, 2, 128, BF), (4, 4, 64, BF), (4, 2, 64, F32)], ids=str)
def test_unseen_keys_and_values_do_not_matter(heads, bad, family):
    """The prompt's later tokens, other branches of a tree, the cache past what a sequence holds, the
    packed neighbours and the tokens nobody selected hold infinities or NaN."""
    dt = heads[3]
    ql = [150, 20, 300]
    q, k, v = make(13, 470, 470, heads[:3], dt)
    ref = A.reference(q, k, v, A.see_prompt(ql, ql), 0.1)
    kb, vb = k.clone(), v.clone()
    cut = 100                      # the end of sequence 0, all of 1, the end of 2
    for t in (kb, vb):
        t[cut:170] = bad
        t[170 + 250:] = bad
    c = i32(A.cu(ql))
    out, lse = K.kpool_attention_prompt(q, kb, vb, c, c, 0.1, return_lse=True, score_kernel=FAMILIES[family])
    keep = list(range(cut)) + list(range(170, 170 + 250))
    A.check(out[keep], lse[keep], [t[keep] for t in ref], "prompt")
    # tree: node 1's branch is broken, nodes 0 and 2 do not see it; the cache ends in garbage
    nodes, prefixes, extents = [3, 1], [200, 90], [300, 170]
    bits = [[0b001, 0b011, 0b101], [0b1]]
    q, k, v = make(14, 4, 470, heads[:3], dt)
    ref = A.reference(q, k, v, A.see_tree(nodes, extents, prefixes, bits), 1.0 / math.sqrt(heads[2]))
    for t in (k, v):
        t[201] = bad
        t[203:300] = bad
        t[300 + 91:] = bad
    _, out, lse, _ = run_tree(nodes, prefixes, extents, bits, heads[:3], dt, family, tensors=(q, k, v))
    keep = [0, 2, 3]
    A.check(out[keep], lse[keep], [t[keep] for t in ref], "tree")
    # selected: everything but the named tokens
    ids = torch.full((4, 70), -1, dtype=torch.int32)
    ids[:, :40] = torch.arange(40) * 2
    q, k, v = make(15, 4, 470, heads[:3], dt)
    ref = A.reference(q, k, v, A.see_selected(ids, [0] * 4, [470]), 0.1)
    for t in (k, v):
        t[1::2] = bad
        t[80:] = bad
    out, lse = K.kpool_attention_selected(q, k, v, ids.cuda(), i32([0, 470]), 0.1, row_seq=i32([0] * 4),
                                          return_lse=True, score_kernel=FAMILIES[family])
    A.check(out, lse, ref, "selected")


@pytest.mark.parametrize("family", FAMILIES)
def test_seen_nan_and_infinite_values_show(family):
    """A value that a row does see reaches it, also in the tiles where other rows do not."""
    ql = [200]
    q, k, v = make(16, 200, 200, (4, 2, 128), BF)
    v[130, 0, 5] = float("nan")
    v[140, 1, 7] = float("inf")
    c = i32([0, 200])
    out, _ = K.kpool_attention_prompt(q, k, v, c, c, 0.05, score_kernel=FAMILIES[family])
    nan = torch.isnan(out)
    assert nan[130:, :2, 5].all() and not nan[:130].any() and nan.sum() == 70 * 2
    inf = torch.isinf(out)
    assert (out[140:, 2:, 7] == float("inf")).all() and not inf[:140].any() and inf.sum() == 60 * 2


@pytest.mark.parametrize("family", FAMILIES)
def test_infinite_keys_give_no_weight(family):
    """A visible key whose score is -inf has weight zero; a row of nothing else counts as empty."""
    q = torch.ones((3, 2, 64), dtype=BF, device="cuda")
    k = torch.zeros((3, 2, 64), dtype=BF, device="cuda")
    v = torch.randn((3, 2, 64), device="cuda").to(BF)
    k[0, :, 0] = -float("inf")
    c = i32([0, 3])
    out, lse = K.kpool_attention_prompt(q, k, v, c, c, 1.0, return_lse=True, score_kernel=FAMILIES[family])
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()
    ref = A.reference(q[1:], torch.zeros_like(k), v, [torch.tensor([1]), torch.tensor([1, 2])], 1.0)
    A.check(out[1:], lse[1:], ref)


def test_no_keys_at_all():
    q, k, v = make(17, 5, 0, (4, 2, 128), BF)
    out, lse = K.kpool_attention_prompt(q, k, v, i32([0, 5]), i32([0, 0]), 0.1, return_lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
    out, lse = K.kpool_attention_selected(q, k, v, i32([[0] * 4] * 5), i32([0, 0]), 0.1, row_seq=i32([0] * 5),
                                          return_lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
    q, k, v = make(17, 0, 5, (4, 2, 128), BF)
    out, lse = K.kpool_attention_prompt(q, k, v, i32([0, 0]), i32([0, 5]), 0.1, return_lse=True)
    assert out.shape == (0, 4, 128)
    q, k, v = make(17, 3, 5, (4, 2, 128), BF)
    out, lse = K.kpool_attention_selected(q, k, v, torch.zeros((3, 0), dtype=torch.int32, device="cuda"), i32([0, 5]),
                                          0.1, row_seq=i32([0] * 3), return_lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("op", ["prompt", "tree", "selected"])
def test_streams_and_graphs_repeat_bit_for_bit(op):
    heads = (8, 2, 128)
    q, k, v = make(18, 60, 3000, heads, BF)
    ws = K.new_attention_workspace(60, 1, *heads, BF)
    out, lse = torch.empty_like(q), torch.empty((60, 8), device="cuda")
    cq, ck, pre = i32([0, 60]), i32([0, 3000]), i32([2900])
    ids = torch.randint(0, 3000, (60, 500), dtype=torch.int32, device="cuda")
    seq = i32([0] * 60)

    def call(stream=None):
        kw = dict(out=out, out_lse=lse, workspace=ws, stream=stream)
        if op == "prompt":
            K.kpool_attention_prompt(q, k, v, cq, ck, 0.1, **kw)
        elif op == "tree":
            K.kpool_attention_tree(q, k, v, cq, ck, pre, 0.1, **kw)
        else:
            K.kpool_attention_selected(q, k, v, ids, ck, 0.1, row_seq=seq, **kw)

    call()
    torch.cuda.synchronize()
    want, wlse = out.clone(), lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        call(side)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out.zero_()
        ws.fill_(0xA5)               # a graph's replay relies on nothing the workspace held
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    q.mul_(0.5)                      # and sees new inputs in the same buffers
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, want)


def test_device_errors_are_reported():
    heads = (4, 2, 128)
    q, k, v = make(19, 6, 40, heads, BF)
    ws = K.new_attention_workspace(6, 2, *heads, BF)
    kw = dict(workspace=ws, return_lse=True)

    def err():
        return K.kpool_last_device_error(ws)
    for cq, ck in (([0, 4, 5], [0, 20, 40]), ([0, 4, 6], [0, 41, 40]), ([1, 4, 6], [0, 20, 40]),
                   ([0, -3, 6], [0, 20, 40]), ([0, 3, 6], [0, 20, 39])):
        K.kpool_attention_prompt(q, k, v, i32(cq), i32(ck), 0.1, **kw)
        assert err() == K.KPOOL_ERR_INVALID_ARG
    K.kpool_attention_prompt(q, k, v, i32([0, 3, 6]), i32([0, 20, 40]), 0.1, **kw)
    assert err() == K.KPOOL_OK
    # a prefix outside its sequence: that sequence's rows are empty, the other's are right
    for pre in ([-1, 7], [18, 7], [2 ** 31 - 1, 7]):
        out, lse = K.kpool_attention_tree(q, k, v, i32([0, 3, 6]), i32([0, 20, 40]), i32(pre), 0.1, **kw)
        assert err() == K.KPOOL_ERR_INVALID_ARG
        assert (out[:3] == 0).all() and torch.isinf(lse[:3]).all()
        ref = A.reference(q[3:], k[20:], v[20:], A.see_tree([3], [20], [7], None), 0.1)
        A.check(out[3:], lse[3:], ref)
    ids = torch.arange(5, dtype=torch.int32, device="cuda").repeat(6, 1)
    seq = i32([0, 1, 2, -1, 1, 0])
    out, lse = K.kpool_attention_selected(q, k, v, ids, i32([0, 20, 40]), 0.1, row_seq=seq, **kw)
    assert err() == K.KPOOL_ERR_INVALID_ARG
    assert (out[2:4] == 0).all() and torch.isinf(lse[2:4]).all() and torch.isfinite(lse[[0, 1, 4, 5]]).all()
