"""Plain 64-bit attention for the tests, and the error each result may have.

A case is described by which keys each query row sees: `see`, a list of 1-D index tensors
(global key tokens, repeats allowed), one per row.
"""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # a rounding is off by at most half a step


def reference(q, k, v, see, scale):
    """(out, lse, out_tol, lse_tol) in float64 on the CPU.

    The tolerances follow from the arithmetic: a score is an fp32 sum of D products (each addition
    rounds, and a matrix unit may truncate instead: 2^-23 of the terms' sum each) and one scaling; an
    error e in an exponent is a relative error e in that weight, in the row's sum and once more through
    the maximum. Weights may be rounded to the input type for the second product, whose sums and the row
    sums are again fp32; out is rounded once.
    """
    dtype = q.dtype
    qd, kd, vd = (t.detach().cpu().double() for t in (q, k, v))
    R, hq, d = qd.shape
    group = hq // kd.shape[1]
    out = torch.zeros((R, hq, d), dtype=torch.float64)
    lse = torch.full((R, hq), -math.inf, dtype=torch.float64)
    tol = torch.zeros((R, hq, d), dtype=torch.float64)
    ltol = torch.zeros((R, hq), dtype=torch.float64)
    for r in range(R):
        j = see[r]
        n = j.numel()
        if n == 0:
            continue
        kr = kd[j].repeat_interleave(group, dim=1)  # [n, Hq, D]
        vr = vd[j].repeat_interleave(group, dim=1)
        s = scale * torch.einsum("hd,nhd->hn", qd[r], kr)
        mag = scale * torch.einsum("hd,nhd->hn", qd[r].abs(), kr.abs()).amax(dim=1)
        z = torch.logsumexp(s, dim=1)
        w = torch.exp(s - z[:, None])
        out[r] = torch.einsum("hn,nhd->hd", w, vr)
        lse[r] = z
        e = (d + 4) * 2.0 ** -23 * mag
        soft = 2 * e + (n + 32) * 2.0 ** -23
        wav = torch.einsum("hn,nhd->hd", w, vr.abs())
        p_round = HALF[dtype] if dtype == torch.bfloat16 else 0.0
        tol[r] = (soft[:, None] + p_round) * wav * 1.01 + HALF[dtype] * out[r].abs() + 1e-30
        ltol[r] = e + (n + 32) * 2.0 ** -23 + 2.0 ** -22 * z.abs()
    return out, lse, tol, ltol


def check(got_out, got_lse, ref, what=""):
    out, lse, tol, ltol = ref
    o = got_out.detach().cpu().double()
    assert torch.isfinite(o).all(), f"{what}: non-finite output"
    over = (o - out).abs() - tol
    assert (over <= 0).all(), f"{what}: out is off by {over.max():.3g} more than it may at {int(over.argmax())}"
    if got_lse is not None:
        z = got_lse.detach().cpu().double()
        empty = torch.isinf(lse)
        assert torch.equal(torch.isinf(z) & (z < 0), empty), f"{what}: wrong empty rows"
        over = torch.where(empty, torch.zeros_like(z), (z - lse).abs() - ltol)
        assert (over <= 0).all(), f"{what}: lse is off by {over.max():.3g} more than it may"


def cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return c


def see_prompt(q_lens, k_lens):
    see, ck = [], cu(k_lens)
    for b, (nq, nk) in enumerate(zip(q_lens, k_lens)):
        for i in range(nq):
            see.append(ck[b] + torch.arange(max(0, min(nk, i + nk - nq + 1))))
    return see


def see_tree(nodes, extents, prefixes, bits):
    """bits: per sequence a list of n ints (bit j: node j is seen), or None for chains."""
    see, ck = [], cu(extents)
    for b, n in enumerate(nodes):
        for i in range(n):
            own = [j for j in range(n) if (bits[b][i] >> j) & 1] if bits else list(range(i + 1))
            see.append(ck[b] + torch.cat([torch.arange(prefixes[b]),
                                          prefixes[b] + torch.tensor(own, dtype=torch.int64)]))
    return see


def see_selected(ids, seq_of_row, k_lens):
    see, ck = [], cu(k_lens)
    for r in range(ids.shape[0]):
        j = ids[r].cpu().long()
        b = seq_of_row[r]
        see.append(ck[b] + j[(j >= 0) & (j < k_lens[b])])
    return see


def mask_words(bits, words):
    """Per-row Python bit sets -> int32 [rows, words]."""
    rows = []
    for x in bits:
        row = []
        for w in range(words):
            u = (x >> (32 * w)) & 0xFFFFFFFF
            row.append(u - (1 << 32) if u >= 1 << 31 else u)
        rows.append(row)
    return torch.tensor(rows, dtype=torch.int32).reshape(len(bits), words)


def random_tree(n, rng):
    """Ancestor bits of a random tree (a forest: about every eighth node is a root)."""
    bits = []
    for i in range(n):
        x = 1 << i
        if i and rng.random() > 0.125:
            x |= bits[rng.randrange(max(0, i - 9), i)]
        bits.append(x)
    return bits
