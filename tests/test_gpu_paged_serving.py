"""Rotary positions, pages and both latent forms together, as the example layers call them."""
import math

import pytest
import torch

from examples import paged_serving as E
from tests import serving_reference as S

pytestmark = pytest.mark.gpu


def test_example_runs():
    whole, again, layer, _ = E.main(tokens=300, steps=2)
    assert torch.isfinite(whole).all() and torch.isfinite(again).all() and layer.pages.lengths == [302]


def test_both_latent_forms_give_the_same_row():
    """The prompt's last row, expanded and absorbed, each against the 64-bit row of what it was given, and the two against
    each other: they differ by the roundings of the projected keys, queries and values to bf16 alone."""
    n = 200
    whole, again, layer, (q, c, kr) = E.main(tokens=n, steps=1)
    nope, half = layer.dims[1], 2.0 ** -8
    k = torch.einsum("nl,hdl->nhd", c.double(), layer.up_k.double())
    v = torch.einsum("nl,hdl->nhd", c.double(), layer.up_v.double())
    keys = torch.cat((k, kr.double()[:, None].expand(-1, layer.heads, -1)), dim=-1)
    row = q[-1].double()
    s = layer.scale * torch.einsum("hd,nhd->hn", row, keys)
    w = torch.softmax(s, dim=-1)
    exact = torch.einsum("hn,nhd->hd", w, v)
    # expanded: k rounds (half a step of every term of a score), v rounds, weights and the result round
    # absorbed: the projected query rounds, the weights, the low result (through |up_v|) and the result
    low = torch.einsum("hd,hdl->hl", row[:, :nope], layer.up_k.double())
    into = layer.scale * torch.einsum("hl,nl->hn", low.abs(), c.double().abs())
    terms = layer.scale * torch.einsum("hd,nhd->hn", row[:, :nope].abs(), k.abs())
    fp32 = 2.0 ** -13 * layer.scale * torch.einsum("hd,nhd->hn", row.abs(), keys.abs())   # 576 additions of 2^-23
    wv = torch.einsum("hn,nhd->hd", w, v.abs())
    back = torch.einsum("hl,hdl->hd", torch.einsum("hn,nl->hl", w, c.double().abs()), layer.up_v.double().abs())
    e1 = (half * terms + fp32).amax(dim=-1, keepdim=True)
    e2 = (half * into + fp32).amax(dim=-1, keepdim=True)
    # (an error e in the scores moves a weight by a factor of at most exp(2 e))
    tol1 = (torch.expm1(2 * e1) + 2 * half) * wv * 1.05 + half * exact.abs()
    tol2 = (torch.expm1(2 * e2) + 2 * half) * back * 1.05 + half * exact.abs()
    assert ((whole[0].double() - exact).abs() <= tol1).all()
    assert ((again[0].double() - exact).abs() <= tol2).all()


def test_grouped_steps_are_one_prompt():
    """A prompt taken whole, and the same tokens as a chunk and single steps: every row within its tolerance."""
    n, cut, heads = 90, 70, (8, 2, 128)
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(h):
        return torch.randn((n, h, 128), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = normal(8), normal(2), normal(2)
    layer = E.GroupedLayer(1, n, *heads)
    parts = [(0, cut)] + [(i, i + 1) for i in range(cut, n)]
    got = torch.cat([layer.step(q[a:b], k[a:b], v[a:b], [b - a]) for a, b in parts])
    pos, freq = torch.arange(n, dtype=torch.int32), S.frequencies(128, 500000.0)
    turned = [S.rotate(t.cpu().double(), pos, freq).to(torch.bfloat16) for t in (q, k)]
    out, _, tol, _ = S.attend(turned[0], turned[1], v.cpu(), [torch.arange(i + 1) for i in range(n)], 1 / math.sqrt(128))
    # rotated channels may round to the other side where they lie between two bf16 values: a step (2^-7) of a term each way
    move = 2 * 2.0 ** -7 * torch.einsum("rhd,nhd->rhn", turned[0].double().abs(),
                                        turned[1].double().abs().repeat_interleave(4, dim=1)).amax(dim=-1) / math.sqrt(128)
    size = v.cpu().double().abs().amax()
    assert ((got.cpu().double() - out).abs() <= tol + torch.expm1(2 * move)[..., None] * size).all()
