"""Refusals of the rotary, paged and latent entry points, the rotary table, and the plain forms of the GPU tests on
cases worked by hand: no GPU, every call comes back before a pointer is used."""
import ctypes
import math

import pytest
import torch

from sparse_attention_kpool_gb300 import build as kbuild
from sparse_attention_kpool_gb300 import kpool as K
from tests import serving_reference as S
from tests.test_attention_devices_host import calls, put  # noqa: F401 (a fixture)

FAKE, BIG = 0x7F0000000000, 1 << 40
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return K.load()


def heads(data=FAKE, ts=1024, hs=576):
    return K.kpool_heads(data, ts, hs)


def pages(data=FAKE, ps=1 << 20, ts=1024, hs=576):
    return K.kpool_pages(data, ps, ts, hs)


def ashape(hq=8, hkv=2, d=128, dtype=K.KPOOL_BF16, scale=0.1, reserved=0):
    return K.kpool_attention_shape(hq, hkv, d, dtype, scale, reserved)


def lshape(h=8, dk=512, dr=64, dv=512, dtype=K.KPOOL_BF16, scale=0.1):
    return K.kpool_latent_shape(h, dk, dr, dv, dtype, scale)


def test_struct_layouts():
    assert [ctypes.sizeof(t) for t in (K.kpool_pages, K.kpool_latent_shape, K.kpool_rotary_part, K.kpool_rotary_shape)] \
        == [32, 24, 64, 16]


# ---------------------------------------------------------------------------- paged

def paged(lib, q=None, k=None, v=None, table=FAKE, max_pages=4, num_pages=9, page=16, lengths=FAKE, cu_q=None, S=3, R=3,
          sh=None, out=None, lse=FAKE, ws=FAKE, ws_bytes=0, opt=None):
    return lib.kpool_attention_paged(q or heads(), k or pages(), v or pages(), table, max_pages, num_pages, page, lengths, cu_q,
                                     S, R, sh or ashape(), out or heads(), lse, ws, ws_bytes, None, opt)


def test_paged_refusals(lib):
    assert paged(lib) == K.KPOOL_ERR_WORKSPACE
    assert paged(lib, cu_q=FAKE, R=9) == K.KPOOL_ERR_WORKSPACE
    bad = [dict(page=0), dict(page=-1), dict(max_pages=-1), dict(num_pages=-1), dict(max_pages=1 << 28, page=16), dict(R=4),
           dict(R=-1), dict(S=-1), dict(table=None), dict(table=FAKE + 2), dict(lengths=None), dict(lengths=FAKE + 1),
           dict(cu_q=FAKE + 2), dict(lse=FAKE + 2), dict(num_pages=1 << 30), dict(S=0, cu_q=FAKE)]
    bad += [dict(sh=ashape(**b)) for b in (dict(hq=7), dict(d=12), dict(scale=0.0), dict(dtype=2), dict(reserved=1))]
    bad += [{w: heads(**b)} for w in ("q", "out") for b in (dict(data=None), dict(data=FAKE + 8), dict(ts=64), dict(hs=577))]
    bad += [{w: pages(**b)} for w in ("k", "v") for b in (dict(data=None), dict(data=FAKE + 8), dict(ps=64), dict(ts=0),
                                                          dict(hs=-576), dict(ps=1 << 40), dict(ts=1025), dict(hs=577))]
    for b in bad:
        assert paged(lib, **b) == K.KPOOL_ERR_INVALID_ARG, b
    for b in (dict(sh=ashape(d=264)), dict(sh=ashape(hq=129, hkv=1)), dict(sh=ashape(dtype=K.KPOOL_F32),
                                                                           opt=K.kpool_options(K.KPOOL_SCORE_TC))):
        assert paged(lib, **b) == K.KPOOL_ERR_UNSUPPORTED, b
    for opt in (K.kpool_options(3), K.kpool_options(0, 1), K.kpool_options(0, 0, None, 0, 0, 1)):
        assert paged(lib, opt=opt) == K.KPOOL_ERR_INVALID_ARG
    n = lib.kpool_attention_workspace_bytes(3, 3, ashape())
    assert paged(lib, ws=None, ws_bytes=BIG) == paged(lib, ws=FAKE + 128, ws_bytes=BIG) == K.KPOOL_ERR_WORKSPACE
    assert paged(lib, ws_bytes=n - 1) == K.KPOOL_ERR_WORKSPACE
    assert paged(lib, R=0, S=0, lengths=None) == K.KPOOL_OK


# --------------------------------------------------------------------------- latent

def latent(lib, q=None, cache=None, table=FAKE, max_pages=4, num_pages=9, page=16, lengths=FAKE, ids=None, width=-1, seq=None,
           S=3, R=3, sh=None, out=None, lse=FAKE, ws=FAKE, ws_bytes=0, opt=None):
    return lib.kpool_attention_latent(q or heads(), cache or pages(), table, max_pages, num_pages, page, lengths, ids, width, seq,
                                      S, R, sh or lshape(), out or heads(), lse, ws, ws_bytes, None, opt)


def test_latent_refusals(lib):
    assert latent(lib) == latent(lib, width=0) == latent(lib, ids=FAKE, width=9) == latent(lib, seq=FAKE, R=7) == K.KPOOL_ERR_WORKSPACE
    bad = [dict(page=0), dict(max_pages=-1), dict(num_pages=-1), dict(max_pages=1 << 28), dict(R=4), dict(R=-1), dict(S=-1),
           dict(table=None), dict(table=FAKE + 2), dict(lengths=None), dict(lengths=FAKE + 1), dict(ids=FAKE + 2, width=4),
           dict(width=4), dict(ids=FAKE, width=-1), dict(width=-2), dict(seq=FAKE + 2), dict(lse=FAKE + 1), dict(S=0, seq=FAKE)]
    bad += [dict(sh=lshape(**b)) for b in (dict(h=0), dict(dk=12, dv=12), dict(dr=0), dict(dr=4), dict(dv=256), dict(dtype=2),
                                           dict(scale=math.nan), dict(scale=-1.0), dict(scale=math.inf))]
    bad += [{w: heads(**b)} for w in ("q", "out") for b in (dict(data=None), dict(data=FAKE + 8), dict(ts=64), dict(hs=577))]
    bad += [dict(cache=pages(**b)) for b in (dict(data=None), dict(data=FAKE + 8), dict(ps=64), dict(ts=0), dict(ts=577),
                                             dict(ps=1 << 40))]
    for b in bad:
        assert latent(lib, **b) == K.KPOOL_ERR_INVALID_ARG, b
    for sh in (lshape(dk=1024, dv=1024), lshape(h=4097)):
        assert latent(lib, sh=sh) == K.KPOOL_ERR_UNSUPPORTED
    tc = K.kpool_options(K.KPOOL_SCORE_TC)
    assert latent(lib, sh=lshape(dtype=K.KPOOL_F32, dk=64, dv=64), opt=tc) == K.KPOOL_ERR_UNSUPPORTED
    assert latent(lib, sh=lshape(dk=256, dv=256), opt=tc) == K.KPOOL_ERR_UNSUPPORTED
    for opt in (K.kpool_options(-1), K.kpool_options(0, 1), K.kpool_options(0, 0, None, 1)):
        assert latent(lib, opt=opt) == K.KPOOL_ERR_INVALID_ARG
    n = lib.kpool_latent_workspace_bytes(3, 3, lshape())
    assert n >= 256 and latent(lib, ws_bytes=n - 1) == latent(lib, ws=None, ws_bytes=BIG) == K.KPOOL_ERR_WORKSPACE
    assert latent(lib, ws=FAKE + 128, ws_bytes=BIG) == K.KPOOL_ERR_WORKSPACE
    assert lib.kpool_latent_workspace_bytes(3, 3, lshape(dv=256)) == lib.kpool_latent_workspace_bytes(-1, 3, lshape()) == 0
    assert latent(lib, R=0, S=0, lengths=None) == K.KPOOL_OK


def latent_prompt(lib, q=None, k=None, kr=None, v=None, cu_q=FAKE, cu_k=FAKE, S=1, R=4, T=9, sh=None, out=None, lse=FAKE, ws=FAKE,
                  ws_bytes=0, opt=None):
    return lib.kpool_attention_latent_prompt(q or heads(), k or heads(), kr or heads(), v or heads(), cu_q, cu_k, S, R, T,
                                             sh or lshape(dk=128, dv=128), out or heads(), lse, ws, ws_bytes, None, opt)


def test_latent_prompt_refusals(lib):
    assert latent_prompt(lib) == K.KPOOL_ERR_WORKSPACE
    bad = [dict(R=-1), dict(T=-1), dict(S=0), dict(cu_q=None), dict(cu_k=None), dict(cu_q=FAKE + 2), dict(cu_k=FAKE + 1),
           dict(lse=FAKE + 2), dict(R=1 << 31)]
    bad += [{w: heads(**b)} for w in ("q", "k", "kr", "v", "out") for b in (dict(data=None), dict(data=FAKE + 8), dict(ts=8),
                                                                            dict(ts=1025))]
    bad += [dict(sh=lshape(**b)) for b in (dict(dk=12), dict(dr=4), dict(dv=4, dk=128), dict(h=0), dict(dk=128, dv=128, scale=0.0))]
    for b in bad:
        assert latent_prompt(lib, **b) == K.KPOOL_ERR_INVALID_ARG, b
    for sh in (lshape(dk=200, dr=64, dv=128), lshape(dk=128, dv=264), lshape(h=4097, dk=128, dv=128)):
        assert latent_prompt(lib, sh=sh) == K.KPOOL_ERR_UNSUPPORTED
    assert latent_prompt(lib, sh=lshape(dk=64, dv=64), opt=K.kpool_options(K.KPOOL_SCORE_TC)) == K.KPOOL_ERR_UNSUPPORTED
    n = lib.kpool_latent_prompt_workspace_bytes(4, 1, lshape(dk=128, dv=128))
    assert latent_prompt(lib, ws_bytes=n - 1) == K.KPOOL_ERR_WORKSPACE
    assert latent_prompt(lib, R=0, cu_q=None, ws=None) == K.KPOOL_OK


# --------------------------------------------------------------------------- rotary

def part(data=FAKE, ts=1024, hs=128, out=FAKE + (1 << 30), ots=1024, ohs=128, h=8, d=128, at=0, reserved=0):
    return K.kpool_rotary_part(K.kpool_heads(data, ts, hs), K.kpool_heads(out, ots, ohs), h, d, at, reserved)


def rotary(lib, q=None, k=None, pos=FAKE, table=FAKE, n=0, rd=64, dtype=K.KPOOL_BF16, flags=0, magnitude=1.0):
    return lib.kpool_rotary(q or part(), k, pos, table, n, K.kpool_rotary_shape(rd, dtype, flags, magnitude), None)


def test_rotary_refusals(lib):
    assert rotary(lib) == rotary(lib, k=part(d=64)) == K.KPOOL_OK      # no tokens: nothing to do
    for b in (dict(n=-1), dict(n=1 << 30), dict(rd=0), dict(rd=63), dict(rd=130), dict(dtype=2), dict(flags=4),
              dict(magnitude=math.inf), dict(magnitude=math.nan), dict(n=3, pos=None), dict(n=3, pos=FAKE + 2),
              dict(n=3, table=None), dict(n=3, table=FAKE + 4)):
        assert rotary(lib, **b) == K.KPOOL_ERR_INVALID_ARG, b
    for b in (dict(h=0), dict(d=0), dict(at=-1), dict(at=65), dict(reserved=1), dict(data=None), dict(data=FAKE + 1), dict(ts=127),
              dict(hs=127), dict(out=None), dict(out=FAKE + 1), dict(ots=1 << 40), dict(ohs=-128),
              dict(out=FAKE, ots=2048)):      # in place, but elsewhere
        assert rotary(lib, q=part(**b), n=3) == rotary(lib, k=part(**b), n=3) == K.KPOOL_ERR_INVALID_ARG, b
    assert rotary(lib, q=part(h=4097)) == rotary(lib, q=part(d=4098, hs=8192, ts=8192)) == K.KPOOL_ERR_UNSUPPORTED


@pytest.mark.parametrize("rd,kw", [(128, {}), (2, {}), (64, dict(base=500000.0, factor=8.0, original_length=8192.0, high=4.0)),
                                   (96, dict(factor=4.0)), (64, dict(factor=40.0, original_length=4096.0))], ids=str)
def test_rotary_table(rd, kw, lib):
    table = K.new_rotary_table(rd, device="cpu", **kw)
    want = S.frequencies(rd, kw.get("base", 10000.0), kw.get("factor", 1.0), kw.get("original_length", 0.0),
                         kw.get("low", 1.0), kw.get("high", 32.0))
    got = torch.tensor([x / 2.0 ** 64 * 2 * math.pi for x in table.tolist()], dtype=torch.float64)
    # a handful of operations in 64 bits on either side, and a power; the table is rounded to 2^-64 of a turn, which is
    # half a step of 2 pi 2^-65 wherever a frequency is below 2^-12 of a turn (above, a double's own steps are larger)
    assert ((got - want).abs() <= 2.0 ** -48 * want + 2 * math.pi * 2.0 ** -65).all()


def test_rotary_table_refusals(lib):
    for args in ((63,), (0,), (64, 0.0), (64, -1.0), (64, math.inf), (64, 1e4, 0.0), (64, 1e4, 2.0, -1.0),
                 (64, 1e4, 2.0, 4096.0, 4.0, 4.0), (64, 1e4, 2.0, 4096.0, -1.0, 4.0), (64, 1e4, math.nan)):
        with pytest.raises(K.KpoolError):
            K.new_rotary_table(*args, device="cpu")


# -------------------------------------------------------------------------- binding

def test_binding_refusals():
    q, kc = torch.zeros((3, 8, 128), dtype=BF), torch.zeros((5, 16, 2, 128), dtype=BF)
    t, n = torch.zeros((3, 4), dtype=I32), torch.zeros(3, dtype=I32)
    for a in ((q, kc, kc[:, :, :1], t, n), (q, kc[0], kc[0], t, n), (q, kc, kc, t[:2], n), (q, kc, kc, t, n[:2]),
              (q[:2], kc, kc, t, n), (q[..., :64], kc, kc, t, n)):
        with pytest.raises(ValueError):
            K.kpool_attention_paged(*a, 0.1)
    with pytest.raises(ValueError):
        K.kpool_attention_paged(q, kc, kc, t, n, 0.1, cu_q=n)
    for a in ((q, kc.float(), kc, t, n), (q.half(), kc.half(), kc.half(), t, n)):
        with pytest.raises(TypeError):
            K.kpool_attention_paged(*a, 0.1)
    with pytest.raises(TypeError):
        K.kpool_attention_paged(q, kc, kc, t, n, 0.1, out=q[:2])
    ql, c = torch.zeros((3, 8, 576), dtype=BF), torch.zeros((5, 16, 576), dtype=BF)
    for a in ((ql, c[..., :500], t, n, 512), (ql, c, t, n, 0), (ql, c, t, n, 576), (ql, c, t[:2], n, 512), (ql[:2], c, t, n, 512)):
        with pytest.raises(ValueError):
            K.kpool_attention_latent(*a, 0.1)
    with pytest.raises(ValueError):
        K.kpool_attention_latent(ql, c, t, n, 512, 0.1, token_ids=t[:2])
    with pytest.raises(ValueError):
        K.kpool_attention_latent(ql, c, t, n, 512, 0.1, row_seq=n[:2])
    with pytest.raises(TypeError):
        K.kpool_attention_latent(ql, c.float(), t, n, 512, 0.1)
    qp, kr = torch.zeros((3, 8, 192), dtype=BF), torch.zeros((9, 64), dtype=BF)
    k, cu = torch.zeros((9, 8, 128), dtype=BF), torch.zeros(2, dtype=I32)
    for a in ((qp, k, kr[:8], k), (qp, k, kr[:, :32], k), (qp, k[:, :7], kr, k), (qp, k, kr, k[:8]), (qp, k, k, k)):
        with pytest.raises(ValueError):
            K.kpool_attention_latent_prompt(*a, cu, cu, 0.1)
    with pytest.raises(ValueError):
        K.kpool_attention_latent_prompt(qp, k, kr, k, cu, cu[:1], 0.1)
    with pytest.raises(TypeError):
        K.kpool_attention_latent_prompt(qp, k, kr.float(), k, cu, cu, 0.1)


def place_all(places, names, made):
    return {n: put(places.get(n, places.get("all", 0)), x) for n, x in zip(names, made)}


def paged_call(places):
    t = place_all(places, ("q", "k", "v", "table", "lengths", "cu_q", "out", "lse", "workspace"),
                  (torch.zeros((3, 4, 64), dtype=BF), torch.zeros((5, 16, 2, 64), dtype=BF), torch.zeros((5, 16, 2, 64), dtype=BF),
                   torch.zeros((3, 4), dtype=I32), torch.zeros(3, dtype=I32), torch.zeros(4, dtype=I32),
                   torch.zeros((3, 4, 64), dtype=BF), torch.zeros((3, 4)), torch.zeros(64, dtype=torch.uint8)))
    K.kpool_attention_paged(t["q"], t["k"], t["v"], t["table"], t["lengths"], 0.1, cu_q=t["cu_q"], out=t["out"], out_lse=t["lse"],
                            workspace=t["workspace"])


def latent_call(places):
    t = place_all(places, ("q", "cache", "table", "lengths", "ids", "seq", "out", "lse", "workspace"),
                  (torch.zeros((3, 4, 80), dtype=BF), torch.zeros((5, 16, 80), dtype=BF), torch.zeros((2, 4), dtype=I32),
                   torch.zeros(2, dtype=I32), torch.zeros((3, 9), dtype=I32), torch.zeros(3, dtype=I32),
                   torch.zeros((3, 4, 64), dtype=BF), torch.zeros((3, 4)), torch.zeros(64, dtype=torch.uint8)))
    K.kpool_attention_latent(t["q"], t["cache"], t["table"], t["lengths"], 64, 0.1, token_ids=t["ids"], row_seq=t["seq"],
                             out=t["out"], out_lse=t["lse"], workspace=t["workspace"])


def latent_prompt_call(places):
    t = place_all(places, ("q", "k", "kr", "v", "cu_q", "cu_k", "out", "lse", "workspace"),
                  (torch.zeros((3, 4, 48), dtype=BF), torch.zeros((5, 4, 32), dtype=BF), torch.zeros((5, 16), dtype=BF),
                   torch.zeros((5, 4, 64), dtype=BF), torch.zeros(2, dtype=I32), torch.zeros(2, dtype=I32),
                   torch.zeros((3, 4, 64), dtype=BF), torch.zeros((3, 4)), torch.zeros(64, dtype=torch.uint8)))
    K.kpool_attention_latent_prompt(t["q"], t["k"], t["kr"], t["v"], t["cu_q"], t["cu_k"], 0.1, out=t["out"], out_lse=t["lse"],
                                    workspace=t["workspace"])


def rotary_call(places):
    t = place_all(places, ("q", "positions", "table", "k", "out", "out_k"),
                  (torch.zeros((3, 4, 64), dtype=BF), torch.zeros(3, dtype=I32), torch.zeros(32, dtype=torch.int64),
                   torch.zeros((3, 1, 64), dtype=BF), torch.zeros((3, 4, 64), dtype=BF), torch.zeros((3, 1, 64), dtype=BF)))
    K.kpool_rotary(t["q"], t["positions"], t["table"], k=t["k"], out_q=t["out"], out_k=t["out_k"])


CALLS = {"kpool_attention_paged": (paged_call, ("q", "k", "v", "table", "lengths", "cu_q", "out", "lse", "workspace")),
         "kpool_attention_latent": (latent_call, ("q", "cache", "table", "lengths", "ids", "seq", "out", "lse", "workspace")),
         "kpool_attention_latent_prompt": (latent_prompt_call, ("q", "k", "kr", "v", "cu_q", "cu_k", "out", "lse", "workspace")),
         "kpool_rotary": (rotary_call, ("q", "positions", "table", "k", "out", "out_k"))}


@pytest.mark.parametrize("where", [1, -1], ids=["other_device", "cpu"])
@pytest.mark.parametrize("name", CALLS)
def test_tensors_elsewhere_are_refused(name, where, calls):  # noqa: F811
    call, tensors = CALLS[name]
    call({})
    assert calls == [name]
    for which in tensors + ("all",):
        with pytest.raises(ValueError):
            call({which: where})
    assert calls == [name]


def test_plain_forms_by_hand():
    """Two keys with scores ln 3 and 0: weights 3/4 and 1/4; a quarter turn in halves and in pairs."""
    q = torch.tensor([[[1.0, 0.0]]] * 2)
    k = torch.tensor([[[math.log(3.0), 5.0]], [[0.0, -2.0]]])
    v = torch.tensor([[[4.0, 0.0, 1.0]], [[0.0, 8.0, 1.0]]])
    out, lse, _, _ = S.attend(q, k, v, [torch.tensor([0, 1]), torch.tensor([], dtype=torch.int64)], 1.0)
    assert torch.allclose(out[:, 0], torch.tensor([[3.0, 2.0, 1.0], [0.0, 0.0, 0.0]], dtype=torch.float64), atol=1e-6)
    assert abs(lse[0, 0] - math.log(4.0)) < 1e-6 and lse[1, 0] == -math.inf
    assert [x.tolist() for x in S.see_paged(torch.tensor([[2, 0], [1, 9]]), [3, 1], 2, [2, 1])] == [[4, 5], [4, 5, 0], [2]]
    assert [x.tolist() for x in S.see_listed(torch.tensor([[2, 0]]), [3], 2, torch.tensor([[2, 7, -1, 0, 2]]), [0])] == [[0, 4, 0]]
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 9.0]]], dtype=torch.float64)
    quarter = torch.tensor([math.pi / 2, 0.0], dtype=torch.float64)
    one = torch.tensor([1])
    assert torch.allclose(S.rotate(x, one, quarter), torch.tensor([[[-3.0, 2.0, 1.0, 4.0, 9.0]]], dtype=torch.float64))
    assert torch.allclose(S.rotate(x, one, quarter, interleaved=True),
                          torch.tensor([[[-2.0, 1.0, 3.0, 4.0, 9.0]]], dtype=torch.float64))
    assert torch.allclose(S.rotate(x, one, quarter, inverse=True, offset=1),
                          torch.tensor([[[1.0, 4.0, 3.0, -2.0, 9.0]]], dtype=torch.float64))
