"""Latent attention on the GPU, absorbed and expanded, against a plain 64-bit implementation through the public
entry points, on both kernel families; the two forms against each other; a layer of all the serving operators."""
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
BIG = (512, 64)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(seed, rows, heads, dims, pages, page, dtype):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((rows, heads, sum(dims)), generator=g) * 1.2).to(dtype).cuda()
    return q, torch.randn((pages, page, sum(dims)), generator=g).to(dtype).cuda()


def run(lengths, page, heads, dims, dtype, family, ids=None, seq=None, seed=1, tensors=None, pool=None, scale=None):
    rows = len(lengths) if seq is None else len(seq)
    total, table = pool or S.pool(lengths, page, random.Random(seed))
    q, cache = tensors or make(seed, rows, heads, dims, total, page, dtype)
    scale = scale or 1.0 / math.sqrt(dims[0] / 4 + dims[1])
    ws = K.new_latent_workspace(rows, len(lengths), heads, *dims, dtype).fill_(0xFF)
    out = torch.full((rows, heads, dims[0]), math.nan, dtype=dtype, device="cuda")
    lse = torch.full((rows, heads), math.nan, device="cuda")
    K.kpool_attention_latent(q, cache, table.cuda(), i32(lengths), dims[0], scale,
                             token_ids=None if ids is None else ids.cuda(), row_seq=None if seq is None else i32(seq),
                             out=out, out_lse=lse, workspace=ws, score_kernel=FAMILIES[family])
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    return (q, cache, table, scale), out, lse


def verify(made, out, lse, lengths, page, ids=None, seq=None, what="", pick=None):
    q, cache, table, scale = made
    seq = list(range(len(lengths))) if seq is None else seq
    if ids is None:
        places = S.slots(table, lengths, page)
        see = [places[b] for b in seq]
    else:
        see = S.see_listed(table, lengths, page, ids, seq)
    if pick is not None:
        q, out, lse, see = q[pick], out[pick], lse[pick], [see[r] for r in pick]
    flat = cache.reshape(-1, 1, cache.shape[2]) if cache.is_contiguous() else cache.flatten(0, 1)[:, None]
    A.check(out, lse, S.attend(q, flat, flat[..., :out.shape[2]], see, scale), what)


SIZES = [(1, BIG, BF), (8, BIG, BF), (16, BIG, BF), (20, BIG, BF), (64, BIG, BF), (65, BIG, BF), (80, BIG, BF),
         (128, BIG, BF), (193, BIG, BF), (4, (64, 16), F32), (9, (128, 32), F32), (3, (24, 8), BF), (2, (960, 64), F32),
         (5, BIG, F32)]


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_whole_caches(size, family):
    heads, dims, dtype = size
    lengths = [1, 130, 0, 64, 257, 63]
    verify(*run(lengths, 16, heads, dims, dtype, family, seed=heads), lengths, 16)


@pytest.mark.parametrize("page", [1, 3, 48, 64, 100, 128, 1000])
@pytest.mark.parametrize("family", FAMILIES)
def test_pages(page, family):
    lengths = [700, 0, 65, 1]
    verify(*run(lengths, page, 16, BIG, BF, family, seed=page), lengths, page)


@pytest.mark.parametrize("lengths,heads", [([20000], 64), ([20000, 3], 128), ([5000, 17, 9000, 0, 300], 16),
                                           ([1500] * 40, 64), ([64] * 300, 32), ([129] * 400, 80), ([12000], 200)], ids=str)
def test_long_caches(lengths, heads):
    """Rows cut over CTAs and joined; the same call twice, bit for bit."""
    made, out, lse = run(lengths, 64, heads, BIG, BF, "auto", seed=3)
    verify(made, out, lse, lengths, 64)
    _, again, alse = run(lengths, 64, heads, BIG, BF, "auto", tensors=made[:2], pool=(None, made[2]))
    assert torch.equal(out, again) and torch.equal(lse, alse)


def test_more_rows_than_the_runs_take():
    lengths = [(i * 5) % 70 for i in range(8500)]
    made, out, lse = run(lengths, 16, 4, BIG, BF, "auto", seed=4)
    verify(made, out, lse, lengths, 16, pick=list(range(0, 8500, 53)))


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("size", [(8, BIG, BF), (64, BIG, BF), (128, BIG, BF), (4, (64, 16), F32)], ids=str)
@pytest.mark.parametrize("width", [1, 20, 64, 131])
def test_lists(width, size, family):
    heads, dims, dtype = size
    lengths, page = [90, 0, 300], 16
    g = torch.Generator().manual_seed(width)
    seq = [0, 2, 2, 0, 2, 0, 2, 1, 0]
    ids = torch.stack([torch.randint(0, max(1, lengths[b]), (width,), generator=g) for b in seq]).to(torch.int32)
    ids[torch.rand(ids.shape, generator=g) < 0.2] = -1
    ids[3] = -1                      # a row without any id
    ids[4, ::2] = 10 ** 9
    ids[5] = 7                       # the same token everywhere
    verify(*run(lengths, page, heads, dims, dtype, family, ids=ids, seq=seq, seed=width), lengths, page, ids, seq)


@pytest.mark.parametrize("rows,width,heads", [(1, 2052, 64), (3, 2052, 128), (16, 2052, 64), (200, 300, 16), (700, 70, 32),
                                              (152, 640, 64), (90, 640, 96)], ids=str)
def test_few_and_many_rows(rows, width, heads):
    """One row spreads over CTAs by its ids, many rows go one by one; bit for bit twice."""
    lengths, page = [4000], 64
    g = torch.Generator().manual_seed(rows)
    ids = torch.stack([torch.randperm(4000, generator=g)[:width] for _ in range(rows)]).to(torch.int32)
    ids[rows // 2, width // 3:] = -1
    seq = [0] * rows
    made, out, lse = run(lengths, page, heads, BIG, BF, "auto", ids=ids, seq=seq, seed=rows)
    verify(made, out, lse, lengths, page, ids, seq, pick=sorted({0, rows // 2, rows - 1, rows // 3}))
    _, again, alse = run(lengths, page, heads, BIG, BF, "auto", ids=ids, seq=seq, tensors=made[:2], pool=(None, made[2]))
    assert torch.equal(out, again) and torch.equal(lse, alse)


@pytest.mark.parametrize("scale", [1e-4, 0.3, 3.0])
def test_scales(scale):
    """Nearly uniform weights, and weights that are all but one zero."""
    lengths = [500, 70]
    verify(*run(lengths, 16, 20, BIG, BF, "auto", seed=6, scale=scale), lengths, 16)


def test_rising_scores():
    """Scores that grow along the tokens move the running maximum at every tile, for some heads only."""
    n, heads = 900, 40
    q, cache = make(7, 1, heads, BIG, 1, n, BF)
    cache = (cache.abs() * (1 + torch.arange(n, device="cuda") / 60)[None, :, None]).to(BF)
    q[:, ::2] = q[:, ::2].abs()
    made, out, lse = run([n], n, heads, BIG, BF, "auto", tensors=(q, cache), pool=(1, torch.zeros((1, 1), dtype=torch.int32)))
    verify(made, out, lse, [n], n)


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_unseen_tokens_do_not_matter(bad, family):
    lengths, page, heads = [150, 20, 0], 48, 16
    total, table = S.pool(lengths, page, random.Random(8))
    q, cache = make(8, 3, heads, BIG, total, page, BF)
    used = torch.cat(S.slots(table, lengths, page)).cuda()
    dirty = torch.full_like(cache, bad)
    dirty.reshape(-1, 576)[used] = cache.reshape(-1, 576)[used]
    made, out, lse = run(lengths, page, heads, BIG, BF, family, tensors=(q, dirty), pool=(total, table))
    verify((q, cache, table, made[3]), out, lse, lengths, page)
    ids = torch.full((3, 70), -1, dtype=torch.int32)
    ids[:, 10:60] = torch.arange(50) * 2
    dirty = torch.full_like(cache, bad)
    named = S.slots(table, lengths, page)[0][:100:2].cuda()
    dirty.reshape(-1, 576)[named] = cache.reshape(-1, 576)[named]
    made, out, lse = run(lengths, page, heads, BIG, BF, family, ids=ids, seq=[0] * 3, tensors=(q, dirty), pool=(total, table))
    verify((q, cache, table, made[3]), out, lse, lengths, page, ids, [0] * 3)


@pytest.mark.parametrize("family", FAMILIES)
def test_tokens_without_weight(family):
    """A visible token whose score is -inf has weight zero; a row of nothing else counts as empty."""
    q = torch.ones((2, 4, 576), dtype=BF, device="cuda")
    cache = torch.randn((2, 16, 576), device="cuda").to(BF) * 0.01
    cache[0, :5, 570] = -math.inf
    table = i32([[0], [0]])
    out, lse = K.kpool_attention_latent(q, cache, table, i32([5, 9]), 512, 0.1, return_lse=True,
                                        score_kernel=FAMILIES[family])
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    flat = cache[0][:, None]
    A.check(out[1:], lse[1:], S.attend(q[1:], flat, flat[..., :512], [torch.arange(5, 9)], 0.1))


@pytest.mark.parametrize("size", [(16, BIG, BF), (4, (64, 16), F32)], ids=str)
def test_strides(size):
    heads, dims, dtype = size
    lengths, page, e, d = [150, 20], 16, sum(dims), dims[0]
    total, table = S.pool(lengths, page, random.Random(9))
    q, cache = make(9, 2, heads, dims, total, page, dtype)
    big = torch.full((total, 2, page + 1, e + 8), math.nan, dtype=dtype, device="cuda")
    big[:, 1, :page, :e] = cache
    qs = torch.full((2, heads + 1, e + 16), math.nan, dtype=dtype, device="cuda")
    qs[:, 1:, 8:8 + e] = q
    guard = torch.full((2, heads + 2, d + 16), 7.0, dtype=dtype, device="cuda")
    out = guard[:, 1:-1, 8:8 + d]
    _, lse = K.kpool_attention_latent(qs[:, 1:, 8:8 + e], big[:, 1, :page, :e], table.cuda(), i32(lengths), d, 0.07, out=out,
                                      return_lse=True)
    verify((q, cache, table, 0.07), out, lse, lengths, page)
    guard[:, 1:-1, 8:8 + d] = 7.0
    assert (guard == 7.0).all(), "wrote outside the output's heads"


@pytest.mark.parametrize("family", FAMILIES)
def test_offsets_past_32_bits(family):
    pages, page, heads = 60000, 64, 8
    cache = torch.empty((pages, page, 576), dtype=BF, device="cuda")
    assert cache.numel() * 2 > 2 ** 32
    q, cache[-9:] = make(10, 2, heads, BIG, 9, page, BF)
    table = torch.tensor([[pages - 1, pages - 3, pages - 5], [pages - 2, pages - 4, pages - 9]], dtype=torch.int32)
    lengths = [130, 190]
    out, lse = K.kpool_attention_latent(q, cache, table.cuda(), i32(lengths), 512, 0.07, return_lse=True,
                                        score_kernel=FAMILIES[family])
    verify((q, cache[-9:], table - (pages - 9), 0.07), out, lse, lengths, page)


def test_nothing_to_see():
    q, cache = make(11, 3, 4, BIG, 4, 16, BF)
    table = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(token_ids=torch.zeros((3, 0), dtype=torch.int32, device="cuda")),
               dict(token_ids=torch.zeros((3, 70), dtype=torch.int32, device="cuda"))):
        out, lse = K.kpool_attention_latent(q, cache, table, i32([0, 0, 0]), 512, 0.1, return_lse=True, **kw)
        assert (out == 0).all() and (lse == -math.inf).all()
    out, lse = K.kpool_attention_latent(q, cache[:0], table, i32([0, 0, 0]), 512, 0.1, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    ids = torch.zeros((3, 0), dtype=torch.int32, device="cuda")
    out, lse = K.kpool_attention_latent(q, cache, table, i32([5, 5, 5]), 512, 0.1, token_ids=ids, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    out, _ = K.kpool_attention_latent(q[:0], cache, table[:0], i32([]), 512, 0.1)
    assert out.shape == (0, 4, 512)


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("listed", [False, True])
def test_device_errors(listed, family):
    page, heads = 16, 8
    q, cache = make(12, 3, heads, BIG, 6, page, BF)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32)
    ids = torch.arange(20, dtype=torch.int32).repeat(3, 1) if listed else None
    ws = K.new_latent_workspace(3, 3, heads, *BIG, BF)

    def call(table, lengths, seq):
        out, lse = K.kpool_attention_latent(q, cache, table.cuda(), i32(lengths), 512, 0.1, return_lse=True, workspace=ws,
                                            token_ids=ids.cuda() if listed else None, row_seq=i32(seq),
                                            score_kernel=FAMILIES[family])
        return out, lse, K.kpool_last_device_error(ws)

    def right(out, lse, pick):
        verify((q, cache, table, 0.1), out, lse, [20, 30, 25], page, ids, [0, 1, 2], pick=pick)
    for n in (33, -1, 2 ** 31 - 1):
        out, lse, err = call(table, [20, n, 25], [0, 1, 2])
        assert err == K.KPOOL_ERR_INVALID_ARG and (out[1] == 0).all() and (lse[1] == -math.inf).all()
        right(out, lse, [0, 2])
    for b in (3, -1, 2 ** 31 - 1):
        out, lse, err = call(table, [20, 30, 25], [0, b, 2])
        assert err == K.KPOOL_ERR_INVALID_ARG and (out[1] == 0).all() and (lse[1] == -math.inf).all()
        right(out, lse, [0, 2])
    for bad in (6, -1, 2 ** 31 - 1):
        t = table.clone()
        t[1, 0] = bad
        out, lse, err = call(t, [20, 30, 25], [0, 1, 2])
        assert err == K.KPOOL_ERR_INVALID_ARG
        right(out, lse, [0, 2])
    out, lse, err = call(table, [20, 30, 25], [0, 1, 2])
    assert err == K.KPOOL_OK
    right(out, lse, None)


@pytest.mark.parametrize("listed", [False, True])
def test_streams_and_graphs(listed):
    page, heads, lengths = 64, 32, [5000, 31, 900]
    total, table = S.pool([n + 64 for n in lengths], page, random.Random(13))
    q, cache = make(13, 3, heads, BIG, total, page, BF)
    ws = K.new_latent_workspace(3, 3, heads, *BIG, BF)
    n, t = i32(lengths), table.cuda()
    ids = torch.arange(200, dtype=torch.int32).repeat(3, 1) * 4 if listed else None
    out, lse = torch.empty((3, heads, 512), dtype=BF, device="cuda"), torch.empty((3, heads), device="cuda")

    def call(stream=None):
        K.kpool_attention_latent(q, cache, t, n, 512, 0.07, token_ids=ids.cuda() if listed else None, out=out, out_lse=lse,
                                 workspace=ws, stream=stream)
    ids = ids.cuda() if listed else None
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
        verify((q, cache, table, 0.07), out, lse, now, page, ids, [0, 1, 2] if listed else None, f"step {step}")
        n.add_(17)


# ------------------------------------------------------------------------- expanded

def prompt(ql, kl, heads, dims, dtype, family="auto", seed=20, tensors=None, scale=None):
    dn, dr, dv = dims
    if tensors is None:
        g = torch.Generator().manual_seed(seed)
        q = (torch.randn((sum(ql), heads, dn + dr), generator=g) * 2).to(dtype).cuda()
        kv = torch.randn((sum(kl), heads, dn + dv), generator=g).to(dtype).cuda()
        tensors = q, kv[..., :dn], torch.randn((sum(kl), dr), generator=g).to(dtype).cuda(), kv[..., dn:]
    q, k, kr, v = tensors
    scale = scale or 1.0 / math.sqrt(dn + dr)
    ws = K.new_latent_prompt_workspace(sum(ql), len(ql), heads, *dims, dtype).fill_(0xFF)
    out = torch.full((sum(ql), heads, dv), math.nan, dtype=dtype, device="cuda")
    lse = torch.full((sum(ql), heads), math.nan, device="cuda")
    K.kpool_attention_latent_prompt(q, k, kr, v, i32(A.cu(ql)), i32(A.cu(kl)), scale, out=out, out_lse=lse, workspace=ws,
                                    score_kernel=FAMILIES[family])
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK
    return (q, k, kr, v, scale), out, lse


def whole_keys(k, kr):
    return torch.cat((k, kr[:, None].expand(-1, k.shape[1], -1)), dim=-1)


FULL = (128, 64, 128)
PACKS = [([1], [1]), ([0, 5, 0, 1, 33], [0, 5, 0, 1, 33]), ([127, 128, 129], [127, 128, 129]),
         ([31, 1, 257], [300, 700, 257]), ([9, 40], [4, 0]), ([300], [300])]


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("size", [(3, FULL, BF), (16, FULL, BF), (2, (64, 32, 64), F32), (3, (32, 16, 40), F32),
                                  (2, (24, 8, 136), BF), (1, (128, 128, 256), F32)], ids=str)
@pytest.mark.parametrize("pack", range(len(PACKS)))
def test_prompts(pack, size, family):
    heads, dims, dtype = size
    ql, kl = PACKS[pack]
    (q, k, kr, v, scale), out, lse = prompt(ql, kl, heads, dims, dtype, family, seed=30 + pack)
    A.check(out, lse, S.attend(q, whole_keys(k, kr), v, A.see_prompt(ql, kl), scale))


@pytest.mark.parametrize("ql,kl,heads", [([700], [700], 8), ([40], [9000], 4), ([300, 1, 64], [2000, 5000, 64], 16),
                                         ([1] * 20, [800] * 20, 4), ([2000], [2000], 2), ([257], [6000], 1),
                                         ([1500, 1, 1], [1500, 1, 1], 16)], ids=str)
def test_longer_prompts(ql, kl, heads):
    """Every split of the work, one and two row tiles per CTA; bit for bit twice."""
    made, out, lse = prompt(ql, kl, heads, FULL, BF)
    q, k, kr, v, scale = made
    see = A.see_prompt(ql, kl)
    pick = sorted(set(range(0, sum(ql), 37)) | {sum(ql) - 1})
    A.check(out[pick], lse[pick], S.attend(q[pick], whole_keys(k, kr), v, [see[r] for r in pick], scale))
    _, again, alse = prompt(ql, kl, heads, FULL, BF, tensors=made[:4])
    assert torch.equal(out, again) and torch.equal(lse, alse)


@pytest.mark.parametrize("family", FAMILIES)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_prompt_unseen_and_seen_values(bad, family):
    ql = [150, 20, 300]
    (q, k, kr, v, scale), want, wlse = prompt(ql, ql, 4, FULL, BF, family)
    ref = S.attend(q, whole_keys(k, kr), v, A.see_prompt(ql, ql), scale)
    kb, vb, rb = k.clone(), v.clone(), kr.clone()
    for t in (kb, vb, rb):
        t[100:170] = bad
        t[170 + 250:] = bad
    _, out, lse = prompt(ql, ql, 4, FULL, BF, family, tensors=(q, kb, rb, vb))
    keep = list(range(100)) + list(range(170, 420))
    A.check(out[keep], lse[keep], [t[keep] for t in ref])
    vb = v.clone()
    vb[130, 1, 5] = bad
    _, out, _ = prompt(ql, ql, 4, FULL, BF, family, tensors=(q, k, kr, vb))
    wild = ~torch.isfinite(out)
    assert wild[130:150, 1, 5].all() and wild.sum() == 20


def test_prompt_strides_and_empty_calls():
    ql, heads = [50, 1, 140], 3
    (q, k, kr, v, scale), want, wlse = prompt(ql, ql, heads, FULL, BF)

    def apart(t):
        return t.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    both = torch.full((191, 64 + 24), math.nan, dtype=BF, device="cuda")
    both[:, 8:72] = kr
    guard = torch.full((191, heads + 2, 128 + 16), 7.0, dtype=BF, device="cuda")
    out = guard[:, 1:-1, 8:136]
    c = i32(A.cu(ql))
    _, lse = K.kpool_attention_latent_prompt(apart(q), apart(k), both[:, 8:72], apart(v), c, c, scale, out=out, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    guard[:, 1:-1, 8:136] = 7.0
    assert (guard == 7.0).all()
    out, lse = K.kpool_attention_latent_prompt(q[:5], k[:0], kr[:0], v[:0], i32([0, 5]), i32([0, 0]), scale, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    out, _ = K.kpool_attention_latent_prompt(q[:0], k, kr, v, i32([0, 0]), i32([0, 191]), scale)
    assert out.shape == (0, heads, 128)


def test_prompt_streams_and_graphs():
    ql, kl, heads = [60, 1], [3000, 500], 4
    (q, k, kr, v, scale), want, wlse = prompt(ql, kl, heads, FULL, BF)
    ws = K.new_latent_prompt_workspace(61, 2, heads, *FULL, BF)
    cq, ck = i32(A.cu(ql)), i32(A.cu(kl))
    out, lse = torch.empty_like(want), torch.empty_like(wlse)

    def call(stream=None):
        K.kpool_attention_latent_prompt(q, k, kr, v, cq, ck, scale, out=out, out_lse=lse, workspace=ws, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        out.fill_(math.nan)
        ws.fill_(0xA5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_prompt_device_errors():
    (q, k, kr, v, scale), want, wlse = prompt([3, 3], [20, 20], 2, FULL, BF)
    ws = K.new_latent_prompt_workspace(6, 2, 2, *FULL, BF)
    for cq, ck in (([0, 4, 5], [0, 20, 40]), ([0, 3, 6], [0, 41, 40]), ([1, 4, 6], [0, 20, 40]), ([0, 3, 6], [0, 20, 39])):
        K.kpool_attention_latent_prompt(q, k, kr, v, i32(cq), i32(ck), scale, workspace=ws)
        assert K.kpool_last_device_error(ws) == K.KPOOL_ERR_INVALID_ARG
    out, _ = K.kpool_attention_latent_prompt(q, k, kr, v, i32([0, 3, 6]), i32([0, 20, 40]), scale, workspace=ws)
    assert K.kpool_last_device_error(ws) == K.KPOOL_OK and torch.equal(out, want)


def test_both_forms_agree():
    """Latents projected to keys and values, against queries projected into the latent space: fp32, where
    nothing is rounded between the two."""
    heads, latent, dn, dr, dv, n = 3, 64, 32, 16, 40, 70
    g = torch.Generator().manual_seed(40)

    def normal(*shape):
        return torch.randn(shape, generator=g).cuda()
    c, kr = normal(n, latent), normal(n, dr)
    q, wk, wv = normal(1, heads, dn + dr), normal(heads, dn, latent) / 8, normal(heads, dv, latent) / 8
    k = torch.einsum("hdl,nl->nhd", wk.double(), c.double()).float()
    v = torch.einsum("hdl,nl->nhd", wv.double(), c.double()).float()
    scale = 1.0 / math.sqrt(dn + dr)
    out, lse = K.kpool_attention_latent_prompt(q, k, kr, v, i32([0, 1]), i32([0, n]), scale, return_lse=True)
    into = torch.cat((torch.einsum("rhd,hdl->rhl", q[..., :dn].double(), wk.double()).float(), q[..., dn:]), dim=-1)
    cache = torch.cat((c, kr), dim=-1)[None]
    low, alse = K.kpool_attention_latent(into, cache, i32([[0]]), i32([n]), latent, scale, return_lse=True)
    back = torch.einsum("rhl,hdl->rhd", low.double(), wv.double())
    # each side within its own tolerance of the same value, and the projections' results rounded to fp32 (2^-24 of
    # the sums of absolute terms, once in the scores and once in the values)
    keys = whole_keys(k, kr)
    _, _, tol, ltol = S.attend(q, keys, v, [torch.arange(n)], scale)
    _, _, ltol2, lltol = S.attend(into, cache[0][:, None], cache[0][:, None, :latent], [torch.arange(n)], scale)
    size = scale * torch.einsum("rhd,hdl,nl->rhn", q[..., :dn].double().abs(), wk.double().abs(), c.double().abs()).amax()
    move = (2 * 2.0 ** -24 * size).cpu()
    spread = torch.einsum("hdl,nl->nhd", wv.double().abs(), c.double().abs()).amax().cpu()
    allowed = tol + torch.einsum("rhl,hdl->rhd", ltol2, wv.double().abs().cpu()) + (2 * move + 2.0 ** -23) * spread
    assert ((back.cpu() - out.cpu().double()).abs() <= allowed).all()
    assert ((lse - alse).cpu().double().abs() <= ltol + lltol + 2 * move).all()
