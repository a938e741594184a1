"""The paged-cache operators as a user calls them, beside their plain form in torch.

Four operators work on one cache of pages: ``append`` (norm and rotation of new queries
and keys, stored with their values), ``attend`` (attention of a chunk of new tokens, one
token included), ``mass`` (the attention weight each entry has received) and ``evict`` (the
lightest entries leave).  ``own`` picks the framework's calls or the plain form.

A case's lengths are a function of the case alone; its values come from the seed.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
DEVICE = "cuda"


# ---- cases ------------------------------------------------------------------------------

def _case(op, seqs, chunk, cached, heads, kv_heads, dim, page, type, ragged=0, **more):
    c = {"op": op, "seqs": seqs, "chunk": chunk, "cached": cached, "heads": heads,
         "kv_heads": kv_heads, "dim": dim, "page": page, "type": type, "ragged": ragged,
         "window": 0}
    if op == "append":
        c.update(input=type, rot=dim, halves=False, norm=True, far=0)
    if op == "mass":
        c.update(decay=1.0)
    if op == "evict":
        c.update(budget=max(1, cached // 2), recent=min(64, cached // 4))
    c.update(more)
    return c


def listed():
    named = [
        # one tick's new rows of a full batch, fp32 as the in-projection leaves them
        ("append_tick", _case("append", 64, 1, 3000, 32, 32, 128, 64, "bf16", 3, input="f32")),
        # a few small chunks of an odd model: partial rotation, positions far beyond the index
        ("append_odd", _case("append", 7, 37, 900, 15, 5, 64, 16, "fp16", 5, rot=32, halves=True,
                             far=1000000)),
        # prompts of several thousand tokens with grouped heads
        ("append_prompt", _case("append", 4, 6000, 9000, 32, 8, 128, 128, "bf16", 7)),
        # one session alone, one token: latency
        ("attend_one", _case("attend", 1, 1, 3000, 32, 32, 128, 64, "bf16")),
        # a tick of a full batch at mixed ages
        ("attend_tick", _case("attend", 64, 1, 3000, 32, 32, 128, 64, "bf16", 11)),
        # a few tokens at a time against long caches with grouped heads
        ("attend_long", _case("attend", 8, 5, 65000, 32, 8, 128, 16, "fp16", 13)),
        # chunks and single tokens in one batch, three heads to a key head, a window
        ("attend_mixed", _case("attend", 12, 700, 5000, 15, 5, 64, 32, "bf16", 17, window=1000)),
        # one long prompt chunk after an earlier one: arithmetic
        ("attend_prompt", _case("attend", 1, 4096, 12000, 32, 8, 128, 128, "bf16")),
        # the weights of a tick
        ("mass_tick", _case("mass", 64, 1, 3000, 32, 32, 128, 64, "bf16", 19)),
        # the weights that the last few hundred tokens of a prompt give to all of it
        ("mass_prompt", _case("mass", 4, 300, 16000, 32, 8, 128, 64, "bf16", 23, decay=0.0)),
        # every session of a batch halves its cache
        ("evict_tick", _case("evict", 16, 0, 3000, 32, 32, 128, 64, "bf16", 29, budget=1500,
                             recent=250)),
        # two long prompts shrink to an eighth and less
        ("evict_prompt", _case("evict", 2, 0, 40000, 32, 8, 128, 16, "fp16", 0, budget=5001,
                               recent=128)),
    ]
    return [dict(c, name=n) for n, c in named]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "mass", "evict"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 5, 8, 16, 32])
    group = rng.choice([1, 1, 2, 3, 4, 7, 8])
    if kv_heads * group > 64:
        group = 1
    page = rng.choice([16, 32, 64, 128, 256])
    type = rng.choice(["bf16", "bf16", "fp16"])
    ragged = rng.randrange(1, 1 << 30) if rng.random() < 0.75 else 0
    entries = 64 * 3000 * 32 * 128 // (kv_heads * dim)     # cache entries of the largest cases
    if op == "append":
        seqs = _spread(rng, 1, 64)
        chunk = _spread(rng, 1, max(1, min(6000, 24000 // seqs, 24000 * 48 // (
            (group + 2) * kv_heads) // seqs)))
        cached = chunk + rng.randrange(0, 3000)
        return _case(op, seqs, chunk, cached, kv_heads * group, kv_heads, dim, page, type, ragged,
                     input=rng.choice([type, type, "f32"]),
                     rot=rng.choice([dim, dim, dim // 2, 2 * rng.randrange(1, dim // 2)]),
                     halves=rng.random() < 0.5, norm=rng.random() < 0.75,
                     far=rng.choice([0, 0, 1000, 2000000]))
    if op == "evict":
        seqs = _spread(rng, 1, 32)
        cached = _spread(rng, 1, max(1, min(60000, entries // 4 // seqs)))
        budget = _spread(rng, 1, cached)
        return _case(op, seqs, 0, cached, kv_heads * group, kv_heads, dim, page, type, ragged,
                     budget=budget, recent=rng.randrange(0, budget + 1))
    seqs = _spread(rng, 1, 64)
    if rng.random() < 0.5:      # single tokens and short chunks, long caches
        chunk = rng.randrange(1, 9)
        cached = _spread(rng, chunk, max(chunk, min(65000, entries // seqs)))
    else:                       # chunks: no more pairs than the largest listed chunk has
        pairs = 4096 * 9000 * 32 // (kv_heads * group)
        cached = _spread(rng, 16, 16000)
        seqs = max(1, min(seqs, entries // cached // 2))
        chunk = _spread(rng, 1, max(1, min(cached, 4096, pairs // cached // seqs)))
    window = rng.choice([0, 0, 0, _spread(rng, 1, cached)])
    more = {"decay": rng.choice([0.0, 0.5, 1.0])} if op == "mass" else {}
    return _case(op, seqs, chunk, cached, kv_heads * group, kv_heads, dim, page, type, ragged,
                 window=window, **more)


def lengths(case):
    """New tokens and cache entries (those included) of each sequence."""
    n, total = [], []
    rng = random.Random(case["ragged"])
    for s in range(case["seqs"]):
        if not case["ragged"]:
            n.append(case["chunk"])
            total.append(case["cached"])
            continue
        c = case["chunk"] and (0 if case["seqs"] > 3 and s == 2 else
                               _spread(rng, 1, case["chunk"]))
        if s == case["seqs"] - 1:
            c = case["chunk"]   # one sequence is as long as the case says
        n.append(c)
        total.append(rng.randrange(c, case["cached"] + 1) if s else case["cached"])
    return n, total


def _visible(case, n, total):
    """Pairs of a new token and an entry that it attends to, and entries that any does."""
    pairs = seen = 0
    w = case["window"] or 1 << 40
    for c, t in zip(n, total):
        if c == 0:
            continue
        first = t - c
        full = max(0, min(c, w - first - 1))            # rows that see all entries up to theirs
        pairs += full * (first + 1) + full * (full - 1) // 2 + (c - full) * w
        seen += min(t, c + w - 1)
    return pairs, seen


def work(case):
    n, total = lengths(case)
    T, H, Hk, D = sum(n), case["heads"], case["kv_heads"], case["dim"]
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "append":
        row = (H + 2 * Hk) * D
        src = 4 if case["input"] == "f32" else 2
        return {"bytes": T * row * (src + size) + T * Hk * 4 + T * 4,
                "flops": T * (H + Hk) * D * 8}
    if case["op"] == "evict":
        kept = sum(min(t, case["budget"]) for t in total)
        return {"bytes": Hk * (sum(total) * 4 + kept * (4 * D * size + 8)),
                "flops": Hk * sum(total)}
    pairs, seen = _visible(case, n, total)
    if case["op"] == "attend":
        return {"bytes": 2 * T * H * D * size + T * H * 4 + 2 * seen * Hk * D * size,
                "flops": 4 * pairs * H * D}
    mass = sum(total) * Hk * (4 if case["decay"] == 0.0 else 8)
    return {"bytes": T * H * (D * size + 4) + seen * Hk * D * size + mass,
            "flops": 2 * pairs * H * D}


# ---- inputs ------------------------------------------------------------------------------

def _normal(g, *shape, scale=1.0, type=torch.float32):
    out = torch.empty(shape, dtype=type, device=DEVICE)
    return out.normal_(generator=g).mul_(scale)


def _pages(case, per_seq, g, perm):
    """A pool with a page to spare and each sequence's pages, in no order."""
    page = case["page"]
    need = [-(-t // page) for t in per_seq]
    order = list(range(sum(need) + 1))
    perm.shuffle(order)
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    return len(order), table.to(DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    perm = random.Random(seed)
    n, total = lengths(case)
    T, H, Hk, D, type = sum(n), case["heads"], case["kv_heads"], case["dim"], TYPES[case["type"]]
    cu = [0]
    for c in n:
        cu.append(cu[-1] + c)
    st = {"case": case, "n": n, "total": total, "at": cu,
          "cu": torch.tensor(cu, dtype=torch.int32, device=DEVICE),
          "len": torch.tensor(total, dtype=torch.int32, device=DEVICE)}
    pool, st["table"] = _pages(case, total, g, perm)
    shape = (pool, Hk, case["page"], D)
    st["k"] = _normal(g, *shape, type=type)
    st["v"] = _normal(g, *shape, type=type)
    st["mass"] = None
    if case["op"] == "append":
        src = TYPES[case["input"]]
        # one row holds a token's queries, keys and values, as a joint projection leaves them
        rows = _normal(g, T, (H + 2 * Hk) * D, scale=2.0, type=src)
        st["q_in"], st["k_in"], st["v_in"] = (
            t.unflatten(1, (-1, D)) for t in rows.split([H * D, Hk * D, Hk * D], 1))
        st["q_alpha"] = 1 + _normal(g, D, scale=0.25) if case["norm"] else None
        st["k_alpha"] = 1 + _normal(g, D, scale=0.25) if case["norm"] else None
        entry = [t - c + i for c, t in zip(n, total) for i in range(c)]
        st["entry"] = torch.tensor(entry, device=DEVICE)
        st["seq"] = torch.tensor([s for s, c in enumerate(n) for _ in range(c)], device=DEVICE)
        st["pos"] = (st["entry"] + case["far"]).int()
        st["mass"] = torch.ones(shape[:3], device=DEVICE)
    elif case["op"] == "evict":
        # weights of very different size, on a grid so that some are equal
        w = _normal(g, *shape[:3], scale=2.0).exp_()
        st["mass"] = w.mul_(64).round_().div_(64)
        kept = [min(t, case["budget"]) for t in total]
        to, st["to_table"] = _pages(case, kept, g, perm)
        for name in "kv":
            st["to_" + name] = torch.zeros((to,) + shape[1:], dtype=type, device=DEVICE)
        st["to_mass"] = torch.zeros((to,) + shape[1:3], device=DEVICE)
    else:
        st["q"] = _normal(g, T, H, D, type=type)
        if case["op"] == "mass":
            st["lse"] = _row_sums(st)
            st["mass"] = _normal(g, *shape[:3]).abs_()
    if own:
        _handles(st)
    return st


def _row_sums(st):
    """The log of each row's softmax sum, which the attention before hands on."""
    case, scale = st["case"], st["case"]["dim"] ** -0.5
    out = torch.empty(st["at"][-1], case["heads"], device=DEVICE)
    for s in range(case["seqs"]):
        a, b = st["at"][s], st["at"][s + 1]
        if a == b:
            continue
        k = _entries(st, st["k"], s).float()
        q = st["q"][a:b].float().transpose(0, 1).unflatten(0, (case["kv_heads"], -1))
        x = torch.matmul(q, k.transpose(-1, -2).unsqueeze(1)).mul_(scale)
        x.masked_fill_(~_mask(st, s), -math.inf)
        out[a:b] = torch.logsumexp(x, -1).flatten(0, 1).transpose(0, 1)
    return out


# ---- the plain form ------------------------------------------------------------------------

def _entries(st, pool, s):
    """Cache entries of sequence s by head: [kv_heads, length, ...]."""
    case = st["case"]
    m = -(-st["total"][s] // case["page"])
    pages = pool[st["table"][s, :m].long()]
    return pages.transpose(0, 1).flatten(1, 2)[:, :st["total"][s]]


def _mask(st, s):
    """True where a new token of sequence s attends to an entry."""
    n, total, w = st["n"][s], st["total"][s], st["case"]["window"]
    at = torch.arange(total - n, total, device=DEVICE)[:, None]
    j = torch.arange(total, device=DEVICE)[None]
    m = j <= at
    return m & (j > at - w) if w else m


def _weights(st, s):
    """Scaled scores of sequence s, masked: [kv_heads, group, new, entries]."""
    case = st["case"]
    a, b = st["at"][s], st["at"][s + 1]
    q = st["q"][a:b].float().transpose(0, 1).unflatten(0, (case["kv_heads"], -1))
    k = _entries(st, st["k"], s).float()
    x = torch.matmul(q, k.transpose(-1, -2).unsqueeze(1)) * case["dim"] ** -0.5
    return x.masked_fill(~_mask(st, s), -math.inf)


def _plain_attend(st):
    case, type = st["case"], st["q"].dtype
    out = torch.empty_like(st["q"])
    lse = torch.empty(st["q"].shape[:2], device=DEVICE)
    for s in range(case["seqs"]):
        a, b = st["at"][s], st["at"][s + 1]
        if a == b:
            continue
        x = _weights(st, s)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p, _entries(st, st["v"], s).float().unsqueeze(1)) / l
        out[a:b] = o.flatten(0, 1).transpose(0, 1).to(type)
        lse[a:b] = (top + torch.log(l)).squeeze(-1).flatten(0, 1).transpose(0, 1)
    return out, lse


def _plain_mass(st):
    case = st["case"]
    mass = st["mass"].clone()
    for s in range(case["seqs"]):
        total = st["total"][s]
        a, b = st["at"][s], st["at"][s + 1]
        lse = st["lse"][a:b].transpose(0, 1).unflatten(0, (case["kv_heads"], -1))
        old = _entries(st, mass, s) * case["decay"] if case["decay"] else 0.0
        new = old + torch.exp(_weights(st, s) - lse.unsqueeze(-1)).sum((1, 2))
        j = torch.arange(total, device=DEVICE)
        mass[st["table"][s].long()[j // case["page"]], :, j % case["page"]] = new.transpose(0, 1)
    return mass


def _plain_turn(st, x, alpha):
    """Norm of each head, then its rotation: [tokens, heads, dim]."""
    case, x = st["case"], x.float()
    if alpha is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * alpha
    rot = case["rot"]
    i = torch.arange(rot // 2, device=DEVICE, dtype=torch.float64)
    angle = st["pos"].double()[:, None] * 10000.0 ** (-2 * i / rot)
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y = x.clone()
    lo, hi = ((slice(0, rot // 2), slice(rot // 2, rot)) if case["halves"] else
              (slice(0, rot, 2), slice(1, rot, 2)))
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., lo] * s + x[..., hi] * c
    return y


def _plain_append(st):
    case, type = st["case"], st["k"].dtype
    q = _plain_turn(st, st["q_in"], st["q_alpha"]).to(type)
    k = _plain_turn(st, st["k_in"], st["k_alpha"]).to(type)
    v = st["v_in"].to(type)
    page = st["table"].long()[st["seq"], st["entry"] // case["page"]]
    row = st["entry"] % case["page"]
    st["k"][page, :, row] = k
    st["v"][page, :, row] = v
    st["mass"][page, :, row] = 0.0
    return q, st["k"], st["v"], st["mass"]


def _plain_evict(st):
    case = st["case"]
    budget, Hk = case["budget"], case["kv_heads"]
    kept = torch.full((case["seqs"], Hk, budget), -1, dtype=torch.int32, device=DEVICE)
    for s in range(case["seqs"]):
        total = st["total"][s]
        m = min(total, budget)
        if m == 0:
            continue
        w = _entries(st, st["mass"], s)
        new = torch.arange(total, device=DEVICE) >= total - case["recent"]
        order = torch.sort(w.masked_fill(new, math.inf), dim=-1, descending=True, stable=True)[1]
        keep = torch.sort(order[:, :m], -1)[0]
        kept[s, :, :m] = keep
        j = torch.arange(m, device=DEVICE)
        page, row = st["to_table"][s].long()[j // case["page"]], j % case["page"]
        head = torch.arange(Hk, device=DEVICE)[:, None]
        for name in ("k", "v", "mass"):
            st["to_" + name][page, :, row] = _entries(st, st[name], s)[head, keep].transpose(0, 1)
    to_len = st["len"].clamp(max=budget)
    return to_len, kept, st["to_k"], st["to_v"], st["to_mass"]


# ---- the framework's calls --------------------------------------------------------------------

def _handles(st):
    import full_duplex_speech_lockstep_gb300 as pp
    st["kv"] = pp.PagedKV(st["k"], st["v"], st["table"], mass=st["mass"])
    if st["case"]["op"] == "evict":
        st["to"] = pp.PagedKV(st["to_k"], st["to_v"], st["to_table"], mass=st["to_mass"])


def _own(st):
    case = st["case"]
    if "kv" not in st:
        _handles(st)
    kv, op = st["kv"], case["op"]
    if op == "append":
        q = kv.append(st["q_in"], st["k_in"], st["v_in"], st["cu"], st["len"],
                      positions=st["pos"], q_alpha=st["q_alpha"], k_alpha=st["k_alpha"],
                      eps=1e-5, rope_base=10000.0, rot_dim=case["rot"], halves=case["halves"])
        return q, st["k"], st["v"], st["mass"]
    if op == "attend":
        return kv.attention(st["q"], st["cu"], st["len"], max_q=case["chunk"],
                            window=case["window"], with_lse=True)
    if op == "mass":
        mass = st["mass"].clone()
        kv.attention_mass(st["q"], st["lse"], st["cu"], st["len"], max_q=case["chunk"],
                          window=case["window"], decay=case["decay"], mass=mass)
        return mass
    to_len, kept = kv.evict(st["len"], case["budget"], case["recent"], st["to"])
    return to_len, kept, st["to_k"], st["to_v"], st["to_mass"]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend, "mass": _plain_mass,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ---- the definition in 64 bits ------------------------------------------------------------------

def _locate(st, table, s, count):
    """Page and row of the first entries of sequence s."""
    page = st["case"]["page"]
    ids = table[s].tolist()
    at = [(ids[j // page], j % page) for j in range(count)]
    return torch.tensor(at, dtype=torch.int64, device=DEVICE).reshape(-1, 2).unbind(1)


def _exact_scores(st, s, head, group, k):
    """Scores of the query heads of one key head in sequence s: [new, group, entries]."""
    case, n, total = st["case"], st["n"][s], st["total"][s]
    a = st["at"][s]
    q = st["q"][a:a + n, head * group:(head + 1) * group].double()
    x = torch.einsum("igd,jd->igj", q, k) / math.sqrt(case["dim"])
    age = (torch.arange(n, device=DEVICE) + (total - n))[:, None, None] - torch.arange(
        total, device=DEVICE)
    hidden = (age < 0) | (age >= (case["window"] or total + 1))
    return x.masked_fill_(hidden, -math.inf)


def exact(case, seed):
    st = prepare(case, seed)
    Hk, D = case["kv_heads"], case["dim"]
    group = case["heads"] // Hk
    if case["op"] == "append":
        rot = case["rot"]
        half = rot // 2
        freq = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(half)],
                            dtype=torch.float64, device=DEVICE)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE),
                           st["pos"].double().outer(freq))[:, None, :]
        new = {}
        for name in "qk":
            x = st[name + "_in"].double()
            if case["norm"]:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5)
                x = x * st[name + "_alpha"].double()
            pair = (x[..., :rot].unflatten(-1, (2, half)).transpose(-1, -2) if case["halves"]
                    else x[..., :rot].unflatten(-1, (half, 2)))
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            z = z.transpose(-1, -2) if case["halves"] else z
            new[name] = torch.cat([z.flatten(-2), x[..., rot:]], -1)
        new["v"] = st["v_in"].double()
        pools = {name: st[name].double() for name in "kv"}
        mass = st["mass"].double()
        for s in range(case["seqs"]):
            a, n = st["at"][s], st["n"][s]
            page, row = (t[st["total"][s] - n:]
                         for t in _locate(st, st["table"], s, st["total"][s]))
            for name in "kv":
                pools[name][page, :, row] = new[name][a:a + n]
            mass[page, :, row] = 0.0
        return new["q"], pools["k"], pools["v"], mass
    if case["op"] == "evict":
        kept = torch.full((case["seqs"], Hk, case["budget"]), -1, dtype=torch.int32)
        to = {n: st["to_" + n].double() for n in ("k", "v", "mass")}
        for s in range(case["seqs"]):
            total = st["total"][s]
            m = min(total, case["budget"])
            page, row = _locate(st, st["table"], s, total)
            to_page, to_row = _locate(st, st["to_table"], s, m)
            for h in range(Hk):
                w = st["mass"][page, h, row].tolist()
                safe = min(case["recent"], total)
                old = sorted(range(total - safe), key=lambda j: (-w[j], j))
                keep = sorted(list(range(total - safe, total)) + old[:m - safe])[:m]
                kept[s, h, :m] = torch.tensor(keep, dtype=torch.int32)
                keep = torch.tensor(keep, dtype=torch.int64, device=DEVICE)
                for name in to:
                    to[name][to_page, h, to_row] = st[name][page[keep], h, row[keep]].double()
        to_len = torch.tensor([min(t, case["budget"]) for t in st["total"]], dtype=torch.int32)
        return to_len.to(DEVICE), kept.to(DEVICE), to["k"], to["v"], to["mass"]
    if case["op"] == "attend":
        out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEVICE)
        lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device=DEVICE)
    else:
        mass = st["mass"].double()
    for s in range(case["seqs"]):
        a, n = st["at"][s], st["n"][s]
        page, row = _locate(st, st["table"], s, st["total"][s])
        for h in range(Hk):
            k = st["k"][page, h, row].double()
            heads = slice(h * group, (h + 1) * group)
            got = torch.zeros(st["total"][s], dtype=torch.float64, device=DEVICE)
            if n:
                x = _exact_scores(st, s, h, group, k)
                if case["op"] == "attend":
                    lse[a:a + n, heads] = torch.logsumexp(x, -1)
                    out[a:a + n, heads] = torch.einsum("igj,jd->igd", torch.softmax(x, -1),
                                                       st["v"][page, h, row].double())
                else:
                    got = torch.exp(x - st["lse"][a:a + n, heads, None].double()).sum((0, 1))
            if case["op"] == "mass":
                old = mass[page, h, row] * case["decay"] if case["decay"] else 0.0
                mass[page, h, row] = old + got
    return (out, lse) if case["op"] == "attend" else mass
