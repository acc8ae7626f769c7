"""Rotary positions on the GPU against the formula in 64 bits."""
import random

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import serving_reference as S

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SCALED = dict(base=500000.0, factor=8.0, original_length=8192.0, low=1.0, high=4.0)


def make(seed, n, heads, dim, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((n, heads, dim), generator=g).to(dtype).cuda()


def far(n, seed=3):
    """Positions over all of int32: the first tokens, a million, the ends of the range, negative ones."""
    rng = random.Random(seed)
    known = [0, 1, 2, 4095, 131071, 1 << 20, 2 ** 31 - 1, -1, -2 ** 31, 10 ** 9 + 7]
    return torch.tensor([known[i] if i < len(known) else rng.randrange(1 << 21) for i in range(n)], dtype=torch.int32)


def freq_of(rd, **kw):
    return S.frequencies(rd, kw.get("base", 10000.0), kw.get("factor", 1.0), kw.get("original_length", 0.0),
                         kw.get("low", 1.0), kw.get("high", 32.0))


def check(got, x, pos, freq, offset=0, interleaved=False, inverse=False, magnitude=1.0):
    want = S.rotate(x.cpu().double(), pos, freq, offset, interleaved, inverse, magnitude)
    tol = S.rotate_tolerance(x.cpu().double(), freq, offset, interleaved, magnitude, x.dtype)
    # far positions: the 64-bit reference's own angle is off by pos 2^-53 of a radian twice over, times |a| + |b|
    own = pos.double().abs()[:, None, None] * 2.0 ** -51 * 2 * x.cpu().double().abs().amax()
    over = (got.cpu().double() - want).abs() - tol - torch.where(tol > 0, own, torch.zeros_like(own))
    assert (over <= 0).all(), f"off by {over.max():.3g} more than it may"


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("q,k,rd,at", [
    ((4, 128), (2, 128), 128, (0, 0)), ((3, 192), (1, 64), 64, (128, 0)), ((2, 80), (1, 80), 32, (0, 48)),
    ((5, 40), (2, 20), 20, (20, 0)), ((1, 2), (1, 3), 2, (0, 1)), ((32, 64), (8, 64), 64, (0, 0)),
    ((7, 96), (1, 104), 96, (0, 8)), ((2, 33), (3, 31), 30, (1, 1)), ((9, 256), None, 16, (16, 0)),
], ids=str)
def test_layouts(q, k, rd, at, interleaved, dtype):
    n = 23
    pos = far(n)
    xq = make(1, n, *q, dtype)
    xk = make(2, n, *k, dtype) if k else None
    table = K.new_rotary_table(rd)
    oq, ok = K.kpool_rotary(xq, pos.cuda(), table, k=xk, q_offset=at[0], k_offset=at[1], interleaved=interleaved)
    check(oq, xq, pos, freq_of(rd), at[0], interleaved)
    if k:
        check(ok, xk, pos, freq_of(rd), at[1], interleaved)
    else:
        assert ok is None


@pytest.mark.parametrize("n", [1, 2, 700, 5000])
@pytest.mark.parametrize("heads", [1, 6, 37])
def test_lengths(n, heads):
    """Few tokens (a head to a thread) and many (eight heads to a thread, the last ones fewer)."""
    pos = torch.arange(n, dtype=torch.int32) + 77
    x = make(n, n, heads, 64, BF)
    out, _ = K.kpool_rotary(x, pos.cuda(), K.new_rotary_table(64))
    check(out, x, pos, freq_of(64))


@pytest.mark.parametrize("inverse", [False, True])
def test_stretched_contexts(inverse):
    pos = far(40)
    x = make(5, 40, 4, 128, F32)
    out, _ = K.kpool_rotary(x, pos.cuda(), K.new_rotary_table(128, **SCALED), inverse=inverse, magnitude=1.37)
    check(out, x, pos, freq_of(128, **SCALED), inverse=inverse, magnitude=1.37)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(interleaved):
    """The inverse is the gradient: the formula's in 64 bits, and differences along random directions."""
    pos, freq = far(9), freq_of(12)
    x = make(6, 9, 3, 20, F32)
    back = make(7, 9, 3, 20, F32)
    table = K.new_rotary_table(12)
    kw = dict(q_offset=4, interleaved=interleaved, magnitude=1.2)
    grad, _ = K.kpool_rotary(back, pos.cuda(), table, inverse=True, **kw)
    leaf = x.cpu().double().requires_grad_()
    S.rotate(leaf, pos, freq, 4, interleaved, False, 1.2).backward(back.cpu().double())
    rotated = leaf.grad.clone()
    check(grad[..., 4:16].contiguous(), back[..., 4:16].contiguous(), pos, freq, 0, interleaved, True, 1.2)
    tol = S.rotate_tolerance(back.cpu().double(), freq, 4, interleaved, 1.2, F32)
    own = pos.double().abs()[:, None, None] * 2.0 ** -50 * back.cpu().abs().amax()
    assert ((grad.cpu().double() - rotated).abs() <= tol + own).all()
    # f is linear: f(x + u) - f(x) = f(u), each call's result within its own tolerance
    u = make(8, 9, 3, 20, F32)
    moved = (K.kpool_rotary(x + u, pos.cuda(), table, **kw)[0] - K.kpool_rotary(x, pos.cuda(), table, **kw)[0]).cpu().double()
    lhs, rhs = (moved * back.cpu().double()).sum(), (u.cpu().double() * grad.cpu().double()).sum()
    size = sum(t.cpu().double().abs() for t in (x, x + u, u)) * back.cpu().double().abs()
    # the copied channels of (x + u) - x round once; the rotated ones as above, every one of |a| + |b| <= 2 max
    assert (lhs - rhs).abs() <= 4 * 2.0 ** -20 * 1.2 * 2 * size.sum()


def test_there_and_back():
    pos = far(30)
    x = make(9, 30, 4, 64, F32)
    table = K.new_rotary_table(64)
    there, _ = K.kpool_rotary(x, pos.cuda(), table)
    again, _ = K.kpool_rotary(there, pos.cuda(), table, inverse=True)
    # the same cosines and sines both ways: c c + s s is 1 within 2^-20, products and sums round
    assert ((again - x).abs() <= 2.0 ** -19 * (x.abs() + x.abs().roll(32, -1))).all()


@pytest.mark.parametrize("dtype,dim,rd,at", [(BF, 128, 128, 0), (BF, 192, 64, 128), (F32, 33, 10, 3)], ids=str)
def test_in_place_and_strides(dtype, dim, rd, at):
    n, heads, pos = 11, 3, far(11)
    x, table = make(10, n, heads, dim, dtype), K.new_rotary_table(rd)
    want, _ = K.kpool_rotary(x, pos.cuda(), table, q_offset=at)
    mine = x.clone()
    got, none = K.kpool_rotary(mine, pos.cuda(), table, q_offset=at, out_q=mine)
    assert got is mine and none is None and torch.equal(mine, want)
    big = torch.full((n + 1, heads + 1, dim + 16), 7.0, dtype=dtype, device="cuda")
    view = big[:n, 1:, 8:8 + dim]
    view.copy_(x)
    first = x.permute(1, 0, 2).contiguous().permute(1, 0, 2)      # heads outermost
    K.kpool_rotary(first, pos.cuda(), table, q_offset=at, out_q=view)
    assert torch.equal(view, want)
    big[:n, 1:, 8:8 + dim] = 7.0
    assert (big == 7.0).all(), "wrote outside the heads"


def test_no_tokens_and_one_head():
    table = K.new_rotary_table(64)
    none = torch.zeros((0, 4, 64), dtype=BF, device="cuda")
    out, _ = K.kpool_rotary(none, torch.zeros(0, dtype=torch.int32, device="cuda"), table)
    assert out.shape == (0, 4, 64)
    x, pos = make(11, 1, 1, 64, BF), torch.tensor([12345], dtype=torch.int32)
    odd = x.as_strided((1, 1, 64), (1, 3, 1))     # strides of single elements carry no meaning
    out, _ = K.kpool_rotary(odd, pos.cuda(), table)
    check(out, x, pos, freq_of(64))


def test_streams_and_graphs():
    x, k, pos = make(12, 50, 8, 128, BF), make(13, 50, 2, 128, BF), far(50).cuda()
    table = K.new_rotary_table(128)
    want, wk = K.kpool_rotary(x, pos, table, k=k)
    oq, ok = torch.empty_like(x), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    K.kpool_rotary(x, pos, table, k=k, out_q=oq, out_k=ok, stream=side)
    side.synchronize()
    assert torch.equal(oq, want) and torch.equal(ok, wk)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kpool_rotary(x, pos, table, k=k, out_q=oq, out_k=ok)
    pos.add_(1)
    g.replay()
    torch.cuda.synchronize()
    again, ak = K.kpool_rotary(x, pos, table, k=k)
    assert torch.equal(oq, again) and torch.equal(ok, ak) and not torch.equal(again, want)


def test_special_values_stay_in_their_pair():
    x, pos = make(14, 6, 2, 64, F32), far(6)
    x[2, 1, 5] = float("nan")
    out, _ = K.kpool_rotary(x, pos.cuda(), K.new_rotary_table(32))
    bad = torch.isnan(out)
    assert bad[2, 1, 5] and bad[2, 1, 21] and bad.sum() == 2
