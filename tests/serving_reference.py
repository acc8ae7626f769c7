"""Plain 64-bit forms of the paged, latent and rotary operators for the tests, and the error each result may have."""
import math

import torch

from tests.attention_reference import HALF


def attend(q, k, v, see, scale):
    """(out, lse, out_tol, lse_tol) in float64: q [R, Hq, E], k [N, Hkv, E], v [N, Hkv, D], see: per row the
    indices into N that it sees (repeats allowed).

    The tolerances follow from the arithmetic, as in attention_reference: a score is an fp32 sum of E products
    (2^-23 of the terms' sum each) and one scaling; an error in an exponent is a relative error in that weight, in
    the row's sum and once more through the maximum. Weights may be rounded to the input type for the second
    product, whose sums and the row sums are again fp32; out is rounded once.
    """
    dtype, dev = q.dtype, q.device
    R, hq, e = q.shape
    hkv, d = k.shape[1], v.shape[2]
    out = torch.zeros((R, hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((R, hq), -math.inf, dtype=torch.float64, device=dev)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(R):
        j = see[r].to(dev)
        n = j.numel()
        if n == 0:
            continue
        qr = q[r].double().reshape(hkv, hq // hkv, e)
        kr, vr = k[j].double(), v[j].double()
        s = scale * torch.einsum("hge,nhe->hgn", qr, kr)
        mag = scale * torch.einsum("hge,nhe->hgn", qr.abs(), kr.abs()).amax(dim=-1)
        z = torch.logsumexp(s, dim=-1)
        w = torch.exp(s - z[..., None])
        err = (e + 4) * 2.0 ** -23 * mag
        soft = 2 * err + (n + 32) * 2.0 ** -23
        wav = torch.einsum("hgn,nhd->hgd", w, vr.abs())
        o = torch.einsum("hgn,nhd->hgd", w, vr)
        p_round = HALF[dtype] if dtype == torch.bfloat16 else 0.0
        out[r] = o.reshape(hq, d)
        lse[r] = z.reshape(hq)
        tol[r] = ((soft[..., None] + p_round) * wav * 1.01 + HALF[dtype] * o.abs() + 1e-30).reshape(hq, d)
        ltol[r] = (err + (n + 32) * 2.0 ** -23 + 2.0 ** -22 * z.abs()).reshape(hq)
    return tuple(t.cpu() for t in (out, lse, tol, ltol))


def slots(table, lengths, page):
    """Per sequence the places of its keys in the flattened pages."""
    out = []
    for b, n in enumerate(lengths):
        j = torch.arange(n)
        out.append(table[b].cpu().long()[j // page] * page + j % page)
    return out


def see_paged(table, lengths, page, q_lens):
    see = []
    for at, n, nq in zip(slots(table, lengths, page), lengths, q_lens):
        see += [at[:max(0, min(n, n - nq + i + 1))] for i in range(nq)]
    return see


def see_listed(table, lengths, page, ids, seq):
    places, see = slots(table, lengths, page), []
    for r in range(ids.shape[0]):
        j = ids[r].cpu().long()
        see.append(places[seq[r]][j[(j >= 0) & (j < lengths[seq[r]])]])
    return see


def pool(lengths, page, rng, spare=2):
    """(pages, table) of a pool in no order; entries behind a sequence's last page are far out of range."""
    need = [(n + page - 1) // page for n in lengths]
    total = sum(need) + spare
    order = list(range(total))
    rng.shuffle(order)
    table = torch.full((len(lengths), max([1] + need)), 2 ** 30, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    return total, table


def frequencies(rotary_dim, base=10000.0, factor=1.0, original=0.0, low=1.0, high=32.0):
    """Radians a token, in 64 bits."""
    f = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    out = []
    for x in f:
        keep = min(1.0, max(0.0, (original * x / (2 * math.pi) - low) / (high - low))) if original else 0.0
        out.append(x * (keep + (1 - keep) / factor))
    return torch.tensor(out, dtype=torch.float64)


def rotate(x, positions, freq, offset=0, interleaved=False, inverse=False, magnitude=1.0):
    """x [T, H, D] in float64, rotated. Differentiable."""
    angle = positions.cpu().double()[:, None] * freq * (-1.0 if inverse else 1.0)
    c, s = (torch.cos(angle) * magnitude)[:, None], (torch.sin(angle) * magnitude)[:, None]
    n = freq.numel()
    head, part, tail = x[..., :offset], x[..., offset:offset + 2 * n], x[..., offset + 2 * n:]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :n], part[..., n:])
    u, v = a * c - b * s, b * c + a * s
    part = torch.stack((u, v), dim=-1).flatten(-2) if interleaved else torch.cat((u, v), dim=-1)
    return torch.cat((head, part, tail), dim=-1)


def rotate_tolerance(x, freq, offset, interleaved, magnitude, dtype):
    """The angle is off by half a step of fp32 below a half turn (2^-25 of it) and the table's rounding, cosine and
    sine by two steps (2^-22 in all with the angle's), and two products and a sum round in fp32: 2^-21 of
    |a| + |b|; the result is rounded once."""
    n = freq.numel()
    size = x.abs().clone()
    part = size[..., offset:offset + 2 * n]
    if interleaved:
        both = (part[..., 0::2] + part[..., 1::2]).repeat_interleave(2, dim=-1)
    else:
        both = (part[..., :n] + part[..., n:]).repeat(1, 1, 2)
    tol = torch.zeros_like(size)
    tol[..., offset:offset + 2 * n] = both * abs(magnitude) * (2.0 ** -21 + HALF[dtype]) + 1e-30
    return tol
