"""Rotary positions, paged caches and latent attention: cases, inputs, plain forms and exact values.

Four operators of one serving layer are described here:

* ``rotary``   positions as rotations of channel pairs of the query and key heads: halves or neighbours
               paired, all of a head or a part of it, frequencies stretched for long contexts;
* ``paged``    attention of each sequence's newest rows (one token, or a chunk) over a key/value cache
               that lies in pages which a table names, with grouped heads;
* ``latent``   attention over one latent vector a token which serves as key (with a rotated part) and as
               value of every head (the absorbed form), in pages: each row over its whole cache, or over
               the token ids that a selection left it;
* ``latent_prompt``  the expanded form for prompts: keys of every head from the latent beside a rotated
               part that all heads share, values of a smaller head size.

Rotation of the channel pair (a, b) number i at position t, f[i] its frequency in radians a token:

    (a cos(t f) - b sin(t f), b cos(t f) + a sin(t f)) * m       (the inverse: -t f)

Attention of a row with visible keys J and query head h:

    s[j] = scale * q[h] . k[j],   out = sum_J exp(s[j]) v[j] / sum_J exp(s[j]),
    lse  = log sum_J exp(s[j]);   J empty gives out = 0 and lse = -inf.
"""
import math

import torch

own = False

KPOOL, TOPK = 4, 2048         # pools and budget of the selections that leave token ids


# ------------------------------------------------------------------------------- cases

def _rotary(dtype, q, k, tokens, start, rotary, **kw):
    """q and k: heads x head size; start: first position of a prompt, or -1 for decode rows at positions of
    their own; the rotated part ends the head when `last`."""
    case = {"op": "rotary", "dtype": dtype, "q_heads": q[0], "q_dim": q[1], "k_heads": k[0], "k_dim": k[1],
            "tokens": tokens, "start": start, "rotary_dim": rotary, "last": False, "interleaved": False,
            "inverse": False, "base": 10000.0, "factor": 1.0, "original": 0.0, "low": 1.0, "high": 32.0,
            "magnitude": 1.0}
    case.update(kw)
    return case


def _paged(dtype, heads, page, q_lens, lengths):
    return {"op": "paged", "dtype": dtype, "q_heads": heads[0], "kv_heads": heads[1], "head_dim": heads[2],
            "page": page, "q_lens": q_lens, "lengths": lengths}


def _latent(dtype, heads, latent, rotary, page, lengths, rows=0, topk=0):
    """rows 0: one row a sequence over its whole cache; else `rows` rows, spread over the sequences in turn,
    over the ids of a selection."""
    return {"op": "latent", "dtype": dtype, "heads": heads, "latent": latent, "rotary": rotary, "page": page,
            "lengths": lengths, "rows": rows, "topk": topk}


def _latent_prompt(dtype, heads, dims, q_lens, k_lens):
    return {"op": "latent_prompt", "dtype": dtype, "heads": heads, "nope": dims[0], "rotary": dims[1],
            "value": dims[2], "q_lens": q_lens, "k_lens": k_lens}


MIXED = "32767,200,17,5000,12345,30001,8191,8192,2,0,24000,16383,999,20480,28111,6553"


def listed():
    return [
        # a decode step of 16 sequences of a long-context model: latency
        dict(_rotary("bf16", (32, 128), (8, 128), 16, -1, 128, base=500000.0, factor=8.0, original=8192.0, high=4.0),
             name="rotary_decode"),
        # a long prompt, whole heads in halves: the memory traffic of q and k
        dict(_rotary("bf16", (32, 128), (8, 128), 32768, 0, 128), name="rotary_prompt"),
        # a chunk of a prompt, the rotated part of latent attention's heads: neighbours paired, behind 128 channels
        dict(_rotary("bf16", (64, 192), (1, 64), 4099, 20000, 64, last=True, interleaved=True, factor=40.0,
                     original=4096.0, magnitude=1.37), name="rotary_latent"),
        # one new chat turn over a short cache, one key head shared
        dict(_paged("bf16", (16, 1, 64), 16, "1", "101"), name="paged_small"),
        # a decode step of 16 sequences of different ages, an empty one among them
        dict(_paged("bf16", (32, 8, 128), 16, ",".join(["1"] * 16), MIXED), name="paged_decode"),
        # a server's mixed step: two chunks of prompts beside decode tokens, larger pages
        dict(_paged("bf16", (32, 8, 128), 64, "512,1,1,200,1,1", "25088,4001,130,10199,16000,9"), name="paged_mixed"),
        # a small shard's decode step: 16 heads over one short and one middling cache
        dict(_latent("bf16", 16, 512, 64, 64, "130,3001"), name="latent_small"),
        # a decode step of 32 sequences, 64 heads over the whole cache
        dict(_latent("bf16", 64, 512, 64, 64, MIXED + "," + MIXED), name="latent_decode"),
        # decode rows after the selection: 16 rows of 64 heads, each over 2052 ids of a long cache
        dict(_latent("bf16", 64, 512, 64, 64, ",".join(["65536"] * 16), rows=16, topk=TOPK), name="latent_selected"),
        # rows of a prompt after their selection, all 128 heads
        dict(_latent("bf16", 128, 512, 64, 64, "16384", rows=512, topk=TOPK), name="latent_selected_rows"),
        # a server's batch of ragged prompts, one of them a later chunk
        dict(_latent_prompt("bf16", 16, (128, 64, 128), "1,517,2048,0,1433,130", "1,517,2048,0,9000,130"),
             name="latent_prompt_packed"),
        # a long document
        dict(_latent_prompt("bf16", 32, (128, 64, 128), "16384", "16384"), name="latent_prompt_long"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(values):
    return ",".join(str(v) for v in values)


def draw(rng):
    op = rng.choice(["rotary", "paged", "latent", "latent_prompt"])
    small = rng.random() < 0.15       # small layers at reference precision
    dtype = "f32" if small else "bf16"
    if op == "rotary":
        rd, qd = rng.choice([(128, 128), (64, 64), (64, 192), (64, 128), (32, 80), (20, 40), (96, 96)])
        q = (rng.choice([1, 8, 12, 32, 64]), qd)
        k = (rng.choice([1, 2, 8]), rng.choice([qd, rd]))
        scaled = rng.random() < 0.5
        start = -1 if rng.random() < 0.4 else _log(rng, 1, 1000000)
        return _rotary(dtype, q, k, _log(rng, 1, 2000 if small else 20000), start, rd, last=rng.random() < 0.5,
                       interleaved=rng.random() < 0.5, inverse=rng.random() < 0.3,
                       base=rng.choice([10000.0, 500000.0, 1000000.0]),
                       factor=rng.choice([2.0, 8.0, 40.0]) if scaled else 1.0,
                       original=rng.choice([0.0, 4096.0, 8192.0]) if scaled else 0.0, high=rng.choice([4.0, 32.0]),
                       magnitude=1.2 if scaled else 1.0)
    if op == "paged":
        heads = rng.choice([(8, 8, 64), (4, 4, 32), (6, 2, 96)] if small else
                           [(32, 8, 128), (32, 8, 128), (16, 1, 64), (8, 8, 128), (24, 4, 64), (12, 2, 128),
                            (64, 1, 128)])
        n = rng.randint(1, 4) if small else _log(rng, 1, 24)
        chunks = rng.random() < 0.4
        q, lens = [], []
        for _ in range(n):
            rows = _log(rng, 1, 16 if small else 500) if chunks and rng.random() < 0.5 else 1
            q.append(rows)
            lens.append(max(rows, _log(rng, 1, 500 if small else 32768)))
        return _paged(dtype, heads, rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256]), _text(q), _text(lens))
    if op == "latent":
        heads = rng.choice([2, 4, 8] if small else [8, 16, 20, 32, 64, 128])
        dims = rng.choice([(64, 16), (128, 32)]) if small else (512, 64)
        page = rng.choice([1, 16, 48, 64, 128])
        if rng.random() < 0.5:
            n = rng.randint(1, 4) if small else _log(rng, 1, 32)
            return _latent(dtype, heads, *dims, page, _text(_log(rng, 1, 500 if small else 32768) for _ in range(n)))
        n = rng.randint(1, 4)
        lens = [_log(rng, 16, 500 if small else 60000) for _ in range(n)]
        topk = KPOOL * (_log(rng, 4, 60) if small else _log(rng, 8, TOPK // KPOOL))
        return _latent(dtype, heads, *dims, page, _text(lens), rows=_log(rng, 1, 64 if small else 400), topk=topk)
    heads = rng.choice([2, 4] if small else [4, 16, 24, 32])
    dims = rng.choice([(32, 16, 32), (64, 32, 64)]) if small else (128, 64, 128)
    q, k = [], []
    for _ in range(rng.randint(1, 5)):
        n = _log(rng, 1, 300 if small else 4000)
        q.append(n)
        k.append(n + (_log(rng, 1, 400 if small else 10000) if rng.random() < 0.4 else 0))
    return _latent_prompt(dtype, heads, dims, _text(q), _text(k))


# ------------------------------------------------------------------------------ inputs

def _ints(text):
    return [int(x) for x in text.split(",")]


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(gen, shape, dtype, factor=1.0):
    """N(0, factor^2), drawn in slices so that a large cache needs no fp32 copy of itself."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // max(1, math.prod(shape[1:])))
    for a in range(0, shape[0], step):
        part = torch.randn((min(step, shape[0] - a),) + tuple(shape[1:]), generator=gen, device="cuda")
        out[a:a + step] = part.mul_(factor).to(dtype)
    return out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(gen, lens, page):
    """(number of pages, page table): the pages of a pool that has been in use for a while, in no order, a
    few of them free; -1 behind a sequence's last one."""
    need = [(n + page - 1) // page for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return total, table


def _selection(gen, pos, pools, topk):
    """Token ids [rows, topk + KPOOL] of rows at positions pos, as a selection leaves them: budget pools in
    rank order (recent ones likelier), expanded, the row's incomplete trailing pool, -1 where empty."""
    budget, rows = topk // KPOOL, pos.numel()
    ids = torch.full((rows, topk + KPOOL), -1, dtype=torch.int32, device="cuda")
    lane = torch.arange(KPOOL, device="cuda", dtype=torch.int64)
    step = max(1, (1 << 26) // max(pools, 1))
    for a in range(0, rows, step):
        p = pos[a:a + step].to(torch.int64)
        n = p.numel()
        eligible = (p + 1) // KPOOL
        if pools:
            at = torch.arange(pools, device="cuda")
            score = torch.rand((n, pools), generator=gen, device="cuda")
            score = score + 0.25 * at / torch.clamp(eligible, min=1)[:, None]
            score.masked_fill_(at[None, :] >= eligible[:, None], -1.0)
            val, idx = torch.topk(score, min(budget, pools), dim=1)
            tok = torch.where((val >= 0)[:, :, None], idx[:, :, None] * KPOOL + lane, -1)
            ids[a:a + n, :tok.shape[1] * KPOOL] = tok.reshape(n, -1).to(torch.int32)
        tail = eligible[:, None] * KPOOL + lane
        ids[a:a + n, topk:] = torch.where(tail <= p[:, None], tail, torch.full_like(tail, -1)).to(torch.int32)
    return ids


def _frequencies(case):
    """Radians a token of each channel pair, in 64 bits: base^(-2i / rotary_dim), divided by factor where a
    pair turns less than `low` times in the original context, as it is from `high` times on, in between
    between; all of them divided where no original context is given."""
    out = []
    for i in range(case["rotary_dim"] // 2):
        f = case["base"] ** (-2.0 * i / case["rotary_dim"])
        keep = 0.0
        if case["original"] > 0:
            turns = case["original"] * f / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - case["low"]) / (case["high"] - case["low"])))
        out.append(f * (keep + (1.0 - keep) / case["factor"]))
    return out


def _prepare_rotary(st, case, gen):
    n, dt = case["tokens"], _dtype(case)
    if case["start"] < 0:
        pos = torch.randint(0, 1 << 20, (n,), generator=gen, device="cuda")
    else:
        pos = torch.arange(case["start"], case["start"] + n, device="cuda")
    st["positions"] = pos.to(torch.int32)
    st["q"] = _normal(gen, (n, case["q_heads"], case["q_dim"]), dt)
    st["k"] = _normal(gen, (n, case["k_heads"], case["k_dim"]), dt)
    rd = case["rotary_dim"]
    st["q_at"] = case["q_dim"] - rd if case["last"] else 0
    st["k_at"] = case["k_dim"] - rd if case["last"] else 0
    st["rd"], st["pairs"], st["inverse"] = rd, case["interleaved"], case["inverse"]
    st["magnitude"] = case["magnitude"]
    st["freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    if own:
        from sparse_attention_kpool_gb300 import kpool
        st["table"] = kpool.new_rotary_table(rd, base=case["base"], factor=case["factor"],
                                             original_length=case["original"], low=case["low"], high=case["high"])
        st["out_q"], st["out_k"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])


def _prepare_paged(st, case, gen):
    hq, hkv, d, dt = case["q_heads"], case["kv_heads"], case["head_dim"], _dtype(case)
    st["ql"], st["kl"], st["page"] = _ints(case["q_lens"]), _ints(case["lengths"]), case["page"]
    total, st["table"] = _pages(gen, st["kl"], case["page"])
    st["lengths"], st["cu_q"] = _i32(st["kl"]), _i32(_cu(st["ql"]))
    st["decode"] = all(n == 1 for n in st["ql"])
    rows = sum(st["ql"])
    st["scale"] = 1.0 / math.sqrt(d)
    # logits of a spread that real layers show: a few keys carry most of a row's weight
    st["q"] = _normal(gen, (rows, hq, d), dt, 2.0)
    st["k"] = _normal(gen, (total, case["page"], hkv, d), dt)
    st["v"] = _normal(gen, (total, case["page"], hkv, d), dt)
    if own:
        from sparse_attention_kpool_gb300 import kpool
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((rows, hq), dtype=torch.float32, device="cuda")
        st["workspace"] = kpool.new_attention_workspace(rows, len(st["kl"]), hq, hkv, d, dt)


def _prepare_latent(st, case, gen):
    h, width, dt = case["heads"], case["latent"] + case["rotary"], _dtype(case)
    st["kl"], st["page"], st["latent"] = _ints(case["lengths"]), case["page"], case["latent"]
    total, st["table"] = _pages(gen, st["kl"], case["page"])
    st["lengths"] = _i32(st["kl"])
    seqs = len(st["kl"])
    rows = case["rows"] or seqs
    st["seq"] = [r % seqs for r in range(rows)]
    st["row_seq"] = st["ids"] = None
    if case["rows"]:
        st["row_seq"] = _i32(st["seq"])
        ids = []
        for b in range(seqs):       # a sequence's rows are its newest tokens
            mine = len(range(b, rows, seqs))
            last = torch.arange(st["kl"][b] - mine, st["kl"][b], device="cuda").clamp(min=0)
            ids.append(_selection(gen, last, st["kl"][b] // KPOOL, case["topk"]))
        st["ids"] = torch.stack([ids[r % seqs][r // seqs] for r in range(rows)])
    # scores are scaled by the size of the unabsorbed keys: three eighths of the latent's for 512 + 64
    st["scale"] = 1.0 / math.sqrt(case["latent"] / 4 + case["rotary"])
    st["q"] = _normal(gen, (rows, h, width), dt, 1.2)
    st["cache"] = _normal(gen, (total, case["page"], width), dt)
    if own:
        from sparse_attention_kpool_gb300 import kpool
        st["out"] = torch.empty((rows, h, case["latent"]), dtype=dt, device="cuda")
        st["lse"] = torch.empty((rows, h), dtype=torch.float32, device="cuda")
        st["workspace"] = kpool.new_latent_workspace(rows, seqs, h, case["latent"], case["rotary"], dt)


def _prepare_latent_prompt(st, case, gen):
    h, dt = case["heads"], _dtype(case)
    dn, dr, dv = case["nope"], case["rotary"], case["value"]
    st["ql"], st["kl"] = _ints(case["q_lens"]), _ints(case["k_lens"])
    st["cu_q"], st["cu_k"] = _i32(_cu(st["ql"])), _i32(_cu(st["kl"]))
    rows, tokens = sum(st["ql"]), sum(st["kl"])
    st["scale"] = 1.0 / math.sqrt(dn + dr)
    st["q"] = _normal(gen, (rows, h, dn + dr), dt, 2.0)
    # keys and values leave their projection side by side, head by head
    kv = _normal(gen, (tokens, h, dn + dv), dt)
    st["k"], st["v"] = kv[..., :dn], kv[..., dn:]
    st["rope"] = _normal(gen, (tokens, dr), dt)
    if own:
        from sparse_attention_kpool_gb300 import kpool
        st["out"] = torch.empty((rows, h, dv), dtype=dt, device="cuda")
        st["lse"] = torch.empty((rows, h), dtype=torch.float32, device="cuda")
        st["workspace"] = kpool.new_latent_prompt_workspace(rows, len(st["kl"]), h, dn, dr, dv, dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"op": case["op"]}
    {"rotary": _prepare_rotary, "paged": _prepare_paged, "latent": _prepare_latent,
     "latent_prompt": _prepare_latent_prompt}[case["op"]](st, case, gen)
    return st


# ------------------------------------------------------------------------- plain forms

def _rotate(x, at, st):
    rd, half = st["rd"], st["rd"] // 2
    angle = st["positions"].double()[:, None] * st["freq"][None, :]   # far positions need 64 bits
    if st["inverse"]:
        angle = -angle
    cos = (torch.cos(angle).float() * st["magnitude"])[:, None, :]
    sin = (torch.sin(angle).float() * st["magnitude"])[:, None, :]
    part = x[..., at:at + rd].float()
    out = x.clone()
    if st["pairs"]:
        a, b = part[..., 0::2], part[..., 1::2]
        out[..., at:at + rd] = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2).to(x.dtype)
    else:
        a, b = part[..., :half], part[..., half:]
        out[..., at:at + rd] = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1).to(x.dtype)
    return out


def _softmax_rows(s, see):
    """Weights exp(s - m) of the seen keys, their sums and the rows' lse; s [..., rows, keys]."""
    if see is not None:
        s = torch.where(see, s, torch.full_like(s, -math.inf))
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    lse = (torch.log(total) + m).squeeze(-1)
    return p, torch.where(total > 0, total, torch.ones_like(total)), lse


def _grouped(q, k, v, scale, see):
    """q [rows, Hq, E], k [keys, Hkv, E] and v [keys, Hkv, D] in fp32, see [rows, keys] -> out [rows, Hq, D], lse."""
    rows, hq, e = q.shape
    hkv, d = k.shape[1], v.shape[2]
    qg = q.reshape(rows, hkv, hq // hkv, e).permute(1, 2, 0, 3).reshape(hkv, -1, e)
    s = torch.matmul(qg, k.permute(1, 2, 0)).reshape(hkv, hq // hkv, rows, -1) * scale
    p, total, lse = _softmax_rows(s, see)
    o = torch.matmul(p.reshape(hkv, -1, p.shape[-1]), v.permute(1, 0, 2)).reshape(hkv, hq // hkv, rows, d) / total
    return o.permute(2, 0, 1, 3).reshape(rows, hq, d), lse.permute(2, 0, 1).reshape(rows, hq)


def _slots(st, b, n):
    """Places of the first n tokens of sequence b in the flattened pages."""
    j = torch.arange(n, device=st["table"].device)
    return st["table"][b, j // st["page"]].long() * st["page"] + j % st["page"]


def _causal(st, keys, out_dim):
    """Rows of every sequence over its keys: keys(b) gives them and their values; rows are the last ones."""
    q = st["q"]
    out = torch.zeros(q.shape[:2] + (out_dim,), dtype=q.dtype, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float32, device=q.device)
    qa = 0
    for b, (nq, nk) in enumerate(zip(st["ql"], st["kl"])):
        if nq and nk:
            k, v = keys(b)
            step = max(1, (1 << 28) // (nk * q.shape[1]))
            for a in range(0, nq, step):
                e = min(nq, a + step)
                top = nk - nq + e
                last = torch.arange(a, e, device=q.device) + (nk - nq)
                see = torch.arange(top, device=q.device)[None, :] <= last[:, None]
                o, z = _grouped(q[qa + a:qa + e].float(), k[:top], v[:top], st["scale"], see)
                out[qa + a:qa + e], lse[qa + a:qa + e] = o.to(out.dtype), z
        qa += nq
    return out, lse


def _plain_paged(st):
    k, v = st["k"].flatten(0, 1), st["v"].flatten(0, 1)

    def keys(b):
        at = _slots(st, b, st["kl"][b])
        return k[at].float(), v[at].float()
    return _causal(st, keys, st["q"].shape[2])


def _plain_latent_prompt(st):
    cu = _cu(st["kl"])
    h = st["q"].shape[1]

    def keys(b):
        at = slice(cu[b], cu[b + 1])
        rope = st["rope"][at].float()[:, None, :].expand(-1, h, -1)
        return torch.cat((st["k"][at].float(), rope), dim=-1), st["v"][at].float()
    return _causal(st, keys, st["v"].shape[2])


def _plain_latent(st):
    q, dl = st["q"], st["latent"]
    rows, h, _ = q.shape
    flat = st["cache"].flatten(0, 1)
    out = torch.zeros((rows, h, dl), dtype=q.dtype, device=q.device)
    lse = torch.full((rows, h), -math.inf, dtype=torch.float32, device=q.device)
    if st["ids"] is None:
        for b, n in enumerate(st["kl"]):
            if n:
                c = flat[_slots(st, b, n)].float()
                s = torch.matmul(q[b].float(), c.t()) * st["scale"]
                p, total, z = _softmax_rows(s, None)
                out[b], lse[b] = (torch.matmul(p, c[:, :dl]) / total).to(out.dtype), z
        return out, lse
    width = st["ids"].shape[1]
    step = max(1, (1 << 27) // (width * flat.shape[1]))
    for a in range(0, rows, step):
        ids = st["ids"][a:a + step].long()
        j = ids.clamp(min=0)
        page = torch.gather(st["table"][st["row_seq"][a:a + step].long()].long(), 1, j // st["page"])
        # (an empty place names page -1 where the sequence has none: any token will do, it is not seen)
        c = flat[(page * st["page"] + j % st["page"]).clamp(min=0)].float()
        s = torch.matmul(q[a:a + step].float(), c.transpose(1, 2)) * st["scale"]
        p, total, z = _softmax_rows(s, (ids >= 0)[:, None, :])
        out[a:a + step], lse[a:a + step] = (torch.matmul(p, c[..., :dl]) / total).to(out.dtype), z
    return out, lse


def run(state):
    st = state
    if own:
        from sparse_attention_kpool_gb300 import kpool
        if st["op"] == "rotary":
            return kpool.kpool_rotary(st["q"], st["positions"], st["table"], k=st["k"], q_offset=st["q_at"],
                                      k_offset=st["k_at"], interleaved=st["pairs"], inverse=st["inverse"],
                                      magnitude=st["magnitude"], out_q=st["out_q"], out_k=st["out_k"])
        kw = {"out": st["out"], "out_lse": st["lse"], "workspace": st["workspace"]}
        if st["op"] == "paged":
            return kpool.kpool_attention_paged(st["q"], st["k"], st["v"], st["table"], st["lengths"], st["scale"],
                                               cu_q=None if st["decode"] else st["cu_q"], **kw)
        if st["op"] == "latent":
            return kpool.kpool_attention_latent(st["q"], st["cache"], st["table"], st["lengths"], st["latent"],
                                                st["scale"], token_ids=st["ids"], row_seq=st["row_seq"], **kw)
        return kpool.kpool_attention_latent_prompt(st["q"], st["k"], st["rope"], st["v"], st["cu_q"], st["cu_k"],
                                                   st["scale"], **kw)
    if st["op"] == "rotary":
        return _rotate(st["q"], st["q_at"], st), _rotate(st["k"], st["k_at"], st)
    return {"paged": _plain_paged, "latent": _plain_latent, "latent_prompt": _plain_latent_prompt}[st["op"]](st)


# ------------------------------------------------------------------------ exact values

def _pairs(case):
    """(query row, key) pairs of one head."""
    if case["op"] == "paged":
        return sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(_ints(case["q_lens"]), _ints(case["lengths"])) if t)
    if case["op"] == "latent_prompt":
        return sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(_ints(case["q_lens"]), _ints(case["k_lens"])))
    lens = _ints(case["lengths"])
    if not case["rows"]:
        return sum(lens)
    total = 0
    for r in range(case["rows"]):
        b, mine = r % len(lens), len(range(r % len(lens), case["rows"], len(lens)))
        at = max(0, lens[b] - mine + r // len(lens))
        total += min(at + 1, case["topk"] + (at + 1) % KPOOL)
    return total


def _dims(case):
    """Heads, and the sizes of a key and of a value."""
    if case["op"] == "paged":
        return case["q_heads"], case["head_dim"], case["head_dim"]
    if case["op"] == "latent":
        return case["heads"], case["latent"] + case["rotary"], case["latent"]
    return case["heads"], case["nope"] + case["rotary"], case["value"]


def _exact_rotary(x, at, case, pos):
    rd = case["rotary_dim"]
    out = x.double()
    for i in range(rd // 2):
        a, b = (at + 2 * i, at + 2 * i + 1) if case["interleaved"] else (at + i, at + rd // 2 + i)
        f = _frequencies(case)[i] * (-1.0 if case["inverse"] else 1.0)
        c = torch.cos(pos.double() * f)[:, None] * case["magnitude"]
        s = torch.sin(pos.double() * f)[:, None] * case["magnitude"]
        u, w = x[..., a].double(), x[..., b].double()
        out[..., a] = u * c - w * s
        out[..., b] = w * c + u * s
    return out


def _exact_rows(q, k, v, scale, first):
    """One head of a sequence in 64 bits: q [n, E] whose row i sees the first `first + i` of k [m, E], v [m, D]."""
    s = (q @ k.t()) * scale
    i = torch.arange(q.shape[0], device=q.device)
    hidden = torch.arange(k.shape[0], device=q.device)[None, :] >= (first + i)[:, None]
    s = s.masked_fill(hidden, -math.inf)
    z = torch.logsumexp(s, dim=-1)
    w = torch.exp(s - torch.where(torch.isinf(z), torch.zeros_like(z), z)[:, None])
    return w @ v, z


def exact(case, seed):
    """What run returns, from the definitions in 64 bits; None where that takes too long."""
    if case["op"] != "rotary":
        heads, e, d = _dims(case)
        if _pairs(case) * heads * 2 * (e + d) > 1.5e12:
            return None
    global own
    mine, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = mine
    if case["op"] == "rotary":
        return (_exact_rotary(st["q"], st["q_at"], case, st["positions"]),
                _exact_rotary(st["k"], st["k_at"], case, st["positions"]))
    dev, rows = st["q"].device, st["q"].shape[0]
    out = torch.zeros((rows, heads, d), dtype=torch.float64, device=dev)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64, device=dev)
    table = st["table"].tolist() if "table" in st else None

    def place(b, tokens):
        return torch.tensor([table[b][t // st["page"]] * st["page"] + t % st["page"] for t in tokens],
                            dtype=torch.int64, device=dev)
    if case["op"] == "latent":
        flat = st["cache"].reshape(-1, e)
        for r in range(rows):
            b = st["seq"][r]
            tokens = range(st["kl"][b]) if st["ids"] is None else [t for t in st["ids"][r].tolist() if t >= 0]
            if not len(tokens):
                continue
            c = flat[place(b, tokens)].double()
            s = st["scale"] * (st["q"][r].double() @ c.t())
            lse[r] = torch.logsumexp(s, dim=-1)
            out[r] = torch.exp(s - lse[r][:, None]) @ c[:, :d]
        return out, lse
    cu_q, cu_k = _cu(st["ql"]), _cu(st["kl"])
    group = heads // (case["kv_heads"] if case["op"] == "paged" else heads)
    for b, (nq, nk) in enumerate(zip(st["ql"], st["kl"])):
        if nq == 0 or nk == 0:
            continue
        at = place(b, range(nk)) if case["op"] == "paged" else torch.arange(cu_k[b], cu_k[b + 1], device=dev)
        for h in range(heads):
            if case["op"] == "paged":
                k = st["k"].flatten(0, 1)[at, h // group].double()
                v = st["v"].flatten(0, 1)[at, h // group].double()
            else:
                k = torch.cat((st["k"][at, h].double(), st["rope"][at].double()), dim=-1)
                v = st["v"][at, h].double()
            for a in range(0, nq, 4096):
                n = min(4096, nq - a)
                where = slice(cu_q[b] + a, cu_q[b] + a + n)
                o, z = _exact_rows(st["q"][where, h].double(), k, v, st["scale"], nk - nq + a + 1)
                out[where, h], lse[where, h] = o, z
    return out, lse


# -------------------------------------------------------------------------------- work

def work(case):
    """What a pass cannot do without: inputs read once (of caches the keys that some row sees), outputs
    written once; the products' operations, six a pair of rotated channels."""
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotary":
        n = case["tokens"]
        channels = n * (case["q_heads"] * case["q_dim"] + case["k_heads"] * case["k_dim"])
        pairs = n * (case["q_heads"] + case["k_heads"]) * (case["rotary_dim"] // 2)
        return {"bytes": 2 * channels * size + n * 4 + case["rotary_dim"] // 2 * 8, "flops": 6 * pairs}
    heads, e, d = _dims(case)
    flops = 2 * (e + d) * _pairs(case) * heads
    if case["op"] == "latent_prompt":
        rows, tokens = sum(_ints(case["q_lens"])), sum(_ints(case["k_lens"]))
        keys = tokens * (heads * (case["nope"] + case["value"]) + case["rotary"])
        return {"bytes": (rows * heads * (e + d) + keys) * size + rows * heads * 4, "flops": flops}
    lens = _ints(case["lengths"])
    pages = sum((n + case["page"] - 1) // case["page"] for n in lens) * 4
    if case["op"] == "paged":
        rows = sum(_ints(case["q_lens"]))
        keys = 2 * sum(lens) * case["kv_heads"] * d
        return {"bytes": (rows * heads * 2 * d + keys) * size + rows * heads * 4 + pages, "flops": flops}
    rows, width = case["rows"] or len(lens), case["topk"] + KPOOL
    tokens, ids = sum(lens), 0
    if case["rows"]:
        ids = rows * width * 4
        tokens = sum(min(n, width * len(range(b, rows, len(lens)))) for b, n in enumerate(lens))
    return {"bytes": (rows * heads * (e + d) + tokens * e) * size + rows * heads * 4 + pages + ids, "flops": flops}
