"""Attention around the KPool selection: cases, inputs, plain forms and exact values.

Three operators of one serving layer are described here:

* ``prompt``    causal attention of a packed batch of query rows over packed keys with
                grouped heads; the queries of a sequence are the last ones of its keys,
                so whole prompts, later chunks of a prompt and single tokens are one form;
* ``tree``      attention of drafted token trees (or chains, or single decode tokens) over
                a key/value cache: every node sees the sequence's committed keys and its own
                ancestors among the drafted ones;
* ``selected``  attention of each row over the token ids a selection left it (index_topk
                ids in pools of kpool, the row's trailing pool, -1 where empty).

For a row with visible keys J and query head h (key head h // (Hq / Hkv))

    s[j] = scale * q[h] . k[j],   out = sum_J exp(s[j]) v[j] / sum_J exp(s[j]),
    lse  = log sum_J exp(s[j]);   J empty gives out = 0 and lse = -inf.
"""
import math

import torch

own = False

HEADS = (32, 8, 128)          # query heads, key heads, head dimension of most cases
MODES = ("prompt", "tree", "selected")


# ------------------------------------------------------------------------------- cases

def _case(op, dtype, heads, **kw):
    return {"op": op, "dtype": dtype, "q_heads": heads[0], "kv_heads": heads[1], "head_dim": heads[2], **kw}


def listed():
    return [
        # the first turn of a chat: one short prompt, where launch latency is what counts
        dict(_case("prompt", "bf16", HEADS, q_lens="37", k_lens="37"), name="prompt_short"),
        # a server's batch of ragged prompts packed together, an empty and a one-token one among them
        dict(_case("prompt", "bf16", HEADS, q_lens="1,517,4096,0,2049,1433,130",
                   k_lens="1,517,4096,0,2049,1433,130"), name="prompt_packed"),
        # two sequences in chunked prefill: the new chunk attends to what the cache holds already
        dict(_case("prompt", "bf16", HEADS, q_lens="512,200", k_lens="25088,10199"), name="prompt_chunk"),
        # a long document as one prompt
        dict(_case("prompt", "bf16", HEADS, q_lens="32768", k_lens="32768"), name="prompt_long"),
        # fp32 reference-precision runs of a small layer
        dict(_case("prompt", "f32", (8, 8, 64), q_lens="300,45", k_lens="300,45"), name="prompt_f32"),
        # one small drafted tree over a short cache, one shared key head
        dict(_case("tree", "bf16", (16, 1, 64), nodes="7", prefixes="100", chain=False), name="tree_small"),
        # a decode step: one token for each of 16 sequences of different ages
        dict(_case("tree", "bf16", HEADS, nodes=",".join(["1"] * 16),
                   prefixes="32767,200,17,5000,12345,30001,8191,8192,2,0,24000,16383,999,20480,28111,6553",
                   chain=True), name="tree_decode"),
        # verification of wide drafts of eight sequences
        dict(_case("tree", "bf16", HEADS, nodes="63,64,40,63,1,17,64,31",
                   prefixes="8191,12000,16500,4099,20000,9001,15000,10240", chain=False), name="tree_verify"),
        # the tiny selection workload's layer: one row, index_topk 16, kpool 4, fp32
        dict(_case("selected", "f32", (4, 4, 32), rows=1, tokens=64, kpool=4, topk=16, decode=True),
             name="selected_tiny"),
        # decode rows of the selection benchmark: 16 rows, each over 2052 ids of a long cache
        dict(_case("selected", "bf16", HEADS, rows=16, tokens=262144, kpool=4, topk=2048, decode=True),
             name="selected_decode"),
        # a packed prompt after its selection: every row attends to the ids it was left
        dict(_case("selected", "bf16", HEADS, rows=4096, tokens=4096, kpool=4, topk=2048, decode=False),
             name="selected_prompt"),
        # the same with one key head shared by all query heads
        dict(_case("selected", "bf16", (64, 1, 128), rows=2048, tokens=16384, kpool=4, topk=2048, decode=True),
             name="selected_shared"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(MODES)
    heads = rng.choice([(32, 8, 128), (32, 8, 128), (16, 1, 64), (8, 8, 128), (24, 4, 64), (12, 2, 128), (64, 1, 128)])
    dtype = "bf16"
    if rng.random() < 0.15:       # small layers at reference precision
        dtype, heads = "f32", rng.choice([(8, 8, 64), (4, 4, 32), (6, 2, 96)])
    small = dtype == "f32"
    if op == "prompt":
        q, k = [], []
        for _ in range(rng.randint(1, 6)):
            n = _log(rng, 1, 400 if small else 6000)
            q.append(n)
            k.append(n + (_log(rng, 1, 400 if small else 16000) if rng.random() < 0.4 else 0))
        return _case(op, dtype, heads, q_lens=",".join(map(str, q)), k_lens=",".join(map(str, k)))
    if op == "tree":
        n = rng.randint(1, 4) if small else _log(rng, 1, 24)
        chain = rng.random() < 0.4
        nodes = [_log(rng, 1, 16 if chain else 64) for _ in range(n)]
        pref = [_log(rng, 1, 500 if small else 32768) for _ in range(n)]
        return _case(op, dtype, heads, nodes=",".join(map(str, nodes)), prefixes=",".join(map(str, pref)), chain=chain)
    kp = rng.choice([1, 3, 4, 4, 8])
    topk = kp * (_log(rng, 4, 60) if small else _log(rng, 16, 2048) // kp + 1)
    decode = rng.random() < 0.5
    rows = _log(rng, 1, 64) if decode else _log(rng, 64, 200 if small else 3000)
    tokens = _log(rng, 64, 500 if small else 100000) if decode else rows
    return _case(op, dtype, heads, rows=rows, tokens=tokens, kpool=kp, topk=topk, decode=decode)


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


def _ancestors(gen, n, width):
    """Bits of a random tree of n nodes in width words of 32: node i sees itself and its parent's bits."""
    u = torch.rand(max(n, 1), generator=gen, device="cuda").tolist()
    rows = []
    for i in range(n):
        bits = 1 << i
        if i > 0:
            parent = int(u[i] * i) if i < 4 else i - 1 - int(u[i] * min(i, 8))
            bits |= rows[parent]
        rows.append(bits)
    words = []
    for bits in rows:
        for w in range(width):
            x = (bits >> (32 * w)) & 0xFFFFFFFF
            words.append(x - (1 << 32) if x >= 1 << 31 else x)
    return words


def _selection(gen, case, pos):
    """Token ids [rows, topk + kpool] of rows at positions pos, as a selection leaves them: budget pools in
    rank order (recent ones likelier), expanded, the row's incomplete trailing pool, -1 where empty."""
    kp, topk = case["kpool"], case["topk"]
    budget, pools = topk // kp, case["tokens"] // kp
    rows = pos.numel()
    ids = torch.full((rows, topk + kp), -1, dtype=torch.int32, device="cuda")
    lane = torch.arange(kp, device="cuda", dtype=torch.int64)
    step = max(1, (1 << 26) // max(pools, 1))
    for a in range(0, rows, step):
        p = pos[a:a + step].to(torch.int64)
        n = p.numel()
        eligible = (p + 1) // kp
        if pools and budget:
            score = torch.rand((n, pools), generator=gen, device="cuda")
            at = torch.arange(pools, device="cuda")
            score = score + 0.25 * at / torch.clamp(eligible, min=1)[:, None]
            score.masked_fill_(at[None, :] >= eligible[:, None], -1.0)
            val, idx = torch.topk(score, min(budget, pools), dim=1)
            tok = idx[:, :, None] * kp + lane
            tok = torch.where((val >= 0)[:, :, None], tok, torch.full_like(tok, -1))
            ids[a:a + n, :tok.shape[1] * kp] = tok.reshape(n, -1).to(torch.int32)
        tail = eligible[:, None] * kp + lane
        ids[a:a + n, topk:] = torch.where(tail <= p[:, None], tail, torch.full_like(tail, -1)).to(torch.int32)
    return ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    dt = _dtype(case)
    st = {"op": case["op"], "scale": 1.0 / math.sqrt(d), "chain": case.get("chain", False)}
    if case["op"] == "prompt":
        st["ql"], st["kl"] = _ints(case["q_lens"]), _ints(case["k_lens"])
        st["cu_q"], st["cu_k"] = _i32(_cu(st["ql"])), _i32(_cu(st["kl"]))
        rows, tokens = sum(st["ql"]), sum(st["kl"])
    elif case["op"] == "tree":
        st["ql"], st["prefix_host"] = _ints(case["nodes"]), _ints(case["prefixes"])
        # each sequence's slot of the cache is larger than what it holds at present
        st["kl"] = [(n + p + 255) // 256 * 256 for n, p in zip(st["ql"], st["prefix_host"])]
        st["cu_q"], st["cu_k"], st["prefix"] = _i32(_cu(st["ql"])), _i32(_cu(st["kl"])), _i32(st["prefix_host"])
        rows, tokens = sum(st["ql"]), sum(st["kl"])
        st["words"] = (max(st["ql"]) + 31) // 32
        st["mask"] = None
        if not case["chain"]:
            words = [w for n in st["ql"] for w in _ancestors(gen, n, st["words"])]
            st["mask"] = _i32(words).reshape(rows, st["words"])
    else:
        rows, tokens = case["rows"], case["tokens"]
        st["cu_k"] = _i32([0, tokens])
        if case["decode"]:
            pos = torch.randint(tokens // 2, tokens, (rows,), generator=gen, device="cuda")
            st["row_seq"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        else:
            pos = torch.arange(rows, device="cuda")
            st["row_seq"] = None
        st["ids"] = _selection(gen, case, pos)
    # logits of a spread that real layers show: a few keys carry most of a row's weight
    st["q"] = _normal(gen, (rows, hq, d), dt, 2.0)
    st["k"] = _normal(gen, (tokens, hkv, d), dt)
    st["v"] = _normal(gen, (tokens, hkv, d), dt)
    if own:
        from sparse_attention_kpool_gb300 import kpool
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((rows, hq), dtype=torch.float32, device="cuda")
        st["workspace"] = kpool.new_attention_workspace(rows, len(st["cu_k"]) - 1, hq, hkv, d, st["q"].dtype)
    return st


# ------------------------------------------------------------------------- plain forms

def _softmax_rows(s, see):
    """Weights exp(s - m) of the seen keys, their sums and the rows' lse; s [..., rows, keys]."""
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    lse = (torch.log(total) + m).squeeze(-1)
    return p, torch.where(total > 0, total, torch.ones_like(total)), lse


def _attend(q, k, v, scale, see):
    """q [rows, Hq, D], k and v [keys, Hkv, D] in fp32, see [rows, keys] -> out [rows, Hq, D], lse [rows, Hq]."""
    rows, hq, d = q.shape
    hkv = k.shape[1]
    qg = q.reshape(rows, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
    s = torch.matmul(qg, k.permute(1, 2, 0)) * scale
    s = s.reshape(hkv, hq // hkv, rows, -1)
    p, total, lse = _softmax_rows(s, see)
    o = torch.matmul(p.reshape(hkv, -1, p.shape[-1]), v.permute(1, 0, 2)).reshape(hkv, hq // hkv, rows, d) / total
    return o.permute(2, 0, 1, 3).reshape(rows, hq, d), lse.permute(2, 0, 1).reshape(rows, hq)


def _plain_rows(st, visible):
    """prompt and tree: sequence by sequence, in chunks of rows that bound the score matrix."""
    q, k, v = st["q"], st["k"], st["v"]
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float32, device=q.device)
    qa = ka = 0
    for b, (nq, nk) in enumerate(zip(st["ql"], st["kl"])):
        live = nk if st["op"] == "prompt" else st["prefix_host"][b] + nq
        kb, vb = k[ka:ka + live].float(), v[ka:ka + live].float()
        step = max(1, (1 << 28) // max(1, live * q.shape[1]))
        for a in range(0, nq, step):
            e = min(nq, a + step)
            top = live - nq + e
            if live == 0 or top <= 0:
                continue
            o, z = _attend(q[qa + a:qa + e].float(), kb[:top], vb[:top], st["scale"], visible(b, qa, a, e, top))
            out[qa + a:qa + e] = o.to(out.dtype)
            lse[qa + a:qa + e] = z
        qa += nq
        ka += nk
    return out, lse


def _plain_prompt(st):
    dev = st["q"].device

    def visible(b, qa, a, e, top):
        last = torch.arange(a, e, device=dev) + (st["kl"][b] - st["ql"][b])
        return torch.arange(top, device=dev)[None, :] <= last[:, None]
    return _plain_rows(st, visible)


def _plain_tree(st):
    dev = st["q"].device

    def visible(b, qa, a, e, top):
        pre = st["prefix_host"][b]
        slot = torch.arange(top, device=dev) - pre
        if st["mask"] is None:
            return slot[None, :] <= torch.arange(a, e, device=dev)[:, None]
        words = st["mask"][qa + a:qa + e].to(torch.int64)
        s = slot.clamp(min=0)
        bit = (words[:, s // 32] >> (s % 32)) & 1
        return (slot < 0)[None, :] | (bit == 1)
    return _plain_rows(st, visible)


def _plain_selected(st):
    q, k, v, ids = st["q"], st["k"], st["v"], st["ids"]
    rows, hq, d = q.shape
    hkv, width = k.shape[1], ids.shape[1]
    out = torch.empty_like(q)
    lse = torch.empty((rows, hq), dtype=torch.float32, device=q.device)
    step = max(1, (1 << 27) // (width * hkv * d))
    for a in range(0, rows, step):
        part = ids[a:a + step].to(torch.int64)
        n = part.shape[0]
        at = part.clamp(min=0).reshape(-1)
        kg = k[at].reshape(n, width, hkv, d).permute(0, 2, 3, 1).float()
        vg = v[at].reshape(n, width, hkv, d).permute(0, 2, 1, 3).float()
        qg = q[a:a + step].float().reshape(n, hkv, hq // hkv, d)
        s = torch.matmul(qg, kg) * st["scale"]
        p, total, z = _softmax_rows(s, (part >= 0)[:, None, None, :])
        out[a:a + step] = (torch.matmul(p, vg) / total).reshape(n, hq, d).to(out.dtype)
        lse[a:a + step] = z.reshape(n, hq)
    return out, lse


def run(state):
    st = state
    if own:
        from sparse_attention_kpool_gb300 import kpool
        kw = {"out": st["out"], "out_lse": st["lse"], "workspace": st["workspace"]}
        if st["op"] == "prompt":
            return kpool.kpool_attention_prompt(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], st["scale"], **kw)
        if st["op"] == "tree":
            return kpool.kpool_attention_tree(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], st["prefix"],
                                              st["scale"], mask=st["mask"], **kw)
        return kpool.kpool_attention_selected(st["q"], st["k"], st["v"], st["ids"], st["cu_k"], st["scale"],
                                              row_seq=st["row_seq"], **kw)
    if st["op"] == "prompt":
        return _plain_prompt(st)
    return _plain_tree(st) if st["op"] == "tree" else _plain_selected(st)


# ------------------------------------------------------------------------ exact values

def _pairs(case):
    """(query row, key slot) pairs of one head."""
    if case["op"] == "prompt":
        return sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(_ints(case["q_lens"]), _ints(case["k_lens"])))
    if case["op"] == "tree":
        return sum(n * p + n * (n + 1) // 2 for n, p in zip(_ints(case["nodes"]), _ints(case["prefixes"])))
    if case["decode"]:
        return case["rows"] * min(case["topk"] + case["kpool"], case["tokens"])
    return sum(min(t + 1, case["topk"] + (t + 1) % case["kpool"]) for t in range(case["rows"]))


def _exact_row(q, k, v, scale):
    """One row in 64 bits: q [Hq, D], its visible keys k, v [n, Hkv, D]."""
    hq, d = q.shape
    if k.shape[0] == 0:
        return q.new_zeros((hq, d)), q.new_full((hq,), -math.inf)
    group = hq // k.shape[1]
    s = scale * torch.einsum("hgd,nhd->hgn", q.reshape(-1, group, d), k)
    z = torch.logsumexp(s, dim=-1)
    return torch.einsum("hgn,nhd->hgd", torch.exp(s - z[..., None]), v).reshape(hq, d), z.reshape(hq)


def exact(case, seed):
    """out and lse from the definition in 64 bits; None where that takes too long."""
    hq, d = case["q_heads"], case["head_dim"]
    if _pairs(case) * hq * d * 4 > 1.5e12:
        return None
    global own
    mine, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = mine
    dev = st["q"].device
    q = st["q"].double()
    rows = q.shape[0]
    out = torch.zeros((rows, hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=dev)
    if case["op"] == "selected":
        for r in range(rows):
            at = st["ids"][r][st["ids"][r] >= 0].long()
            out[r], lse[r] = _exact_row(q[r], st["k"][at].double(), st["v"][at].double(), st["scale"])
        return out, lse
    cu_q, cu_k = _cu(st["ql"]), _cu(st["kl"])
    group = hq // case["kv_heads"]
    for b, nq in enumerate(st["ql"]):
        pre = st["kl"][b] - nq if case["op"] == "prompt" else st["prefix_host"][b]
        n = pre + nq
        if n <= 0 or nq == 0:
            continue
        see = torch.zeros((nq, n), dtype=torch.bool, device=dev)
        if case["op"] == "prompt" or case["chain"]:
            see |= torch.ones((nq, n), dtype=torch.bool, device=dev).tril(diagonal=pre)
        else:
            see[:, :pre] = True
            words = st["mask"][cu_q[b]:cu_q[b + 1]].tolist()
            for i in range(nq):
                for j in range(nq):
                    see[i, pre + j] = (words[i][j // 32] >> (j % 32)) & 1 == 1
        for g in range(case["kv_heads"]):
            kb = st["k"][cu_k[b]:cu_k[b] + n, g].double()
            vb = st["v"][cu_k[b]:cu_k[b] + n, g].double()
            for h in range(g * group, (g + 1) * group):
                for a in range(0, nq, 4096):
                    e = min(nq, a + 4096)
                    s = (q[cu_q[b] + a:cu_q[b] + e, h] @ kb.t()) * st["scale"]
                    s[~see[a:e]] = -math.inf
                    z = torch.logsumexp(s, dim=-1, keepdim=True)
                    some = see[a:e].any(dim=-1, keepdim=True)
                    w = torch.where(some, torch.exp(s - z), torch.zeros_like(s))
                    out[cu_q[b] + a:cu_q[b] + e, h] = w @ vb
                    lse[cu_q[b] + a:cu_q[b] + e, h] = z.squeeze(-1)
    return out, lse


# -------------------------------------------------------------------------------- work

def work(case):
    """q, the visible keys and values and the ids or masks read once, out and lse written once; two products."""
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    e = 2 if case["dtype"] == "bf16" else 4
    extra = 0
    if case["op"] == "prompt":
        rows, keys = sum(_ints(case["q_lens"])), sum(_ints(case["k_lens"]))
    elif case["op"] == "tree":
        nodes = _ints(case["nodes"])
        rows, keys = sum(nodes), sum(nodes) + sum(_ints(case["prefixes"]))
        extra = 0 if case["chain"] else rows * ((max(nodes) + 31) // 32) * 4
    else:
        rows = case["rows"]
        width = case["topk"] + case["kpool"]
        keys = min(case["tokens"], rows * width)
        extra = rows * width * 4
    nbytes = 2 * rows * hq * d * e + rows * hq * 4 + 2 * keys * hkv * d * e + extra
    return {"bytes": nbytes, "flops": 4 * _pairs(case) * hq * d}
