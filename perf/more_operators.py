"""The 8-bit paged cache and the log probabilities of given tokens as a user calls them, beside
their plain forms in torch.

``append`` (norm and rotation of new queries and keys, stored with their values in 8 bits),
``attend`` (attention of new tokens over such a cache), ``read`` (entries back into a cache of 16
bits) and ``score`` (log probabilities of given tokens, entropy, top alternatives).  ``own`` picks
the framework's calls or the plain form.

An entry of a key head is one row of e4m3 codes and one power of two: with a = max |y| and e the
least whole number such that a 2^-e <= 448 (-127 at least), the codes are y 2^-e rounded to e4m3
and the scale is 2^e, held as the byte e + 127.

A case's lengths are a function of the case alone; its values come from the seed.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DEVICE = "cuda"


# ---- cases ------------------------------------------------------------------------------

def _cache(op, seqs, chunk, cached, heads, kv_heads, dim, page, type, ragged=0, **more):
    c = {"op": op, "seqs": seqs, "chunk": chunk, "cached": cached, "heads": heads,
         "kv_heads": kv_heads, "dim": dim, "page": page, "type": type, "ragged": ragged,
         "window": 0}
    if op == "append":
        c.update(input=type, rot=dim, halves=False, norm=True, far=0)
    c.update(more)
    return c


def _score(rows, inner, n, type, top, entropy=True, pad=0, spread=3.0):
    return {"op": "score", "rows": rows, "inner": inner, "n": n, "type": type, "top": top,
            "entropy": entropy, "pad": pad, "spread": spread}


def listed():
    named = [
        # one tick's new rows of a full batch, fp32 as the in-projection leaves them
        ("append_tick", _cache("append", 64, 1, 3000, 32, 32, 128, 64, "bf16", 3, input="f32")),
        # prompts of several thousand tokens with grouped heads
        ("append_prompt", _cache("append", 4, 6000, 9000, 32, 8, 128, 128, "bf16", 7)),
        # one session alone, one token: latency
        ("attend_one", _cache("attend", 1, 1, 3000, 32, 32, 128, 64, "bf16")),
        # a tick of a full batch at mixed ages
        ("attend_tick", _cache("attend", 64, 1, 3000, 32, 32, 128, 64, "bf16", 11)),
        # a few tokens at a time against long caches with grouped heads
        ("attend_long", _cache("attend", 8, 5, 65000, 32, 8, 128, 16, "fp16", 13)),
        # chunks of up to a few hundred tokens of an odd model, three heads to a key head, a window
        ("attend_mixed", _cache("attend", 12, 300, 5000, 15, 5, 64, 32, "bf16", 17, window=1000)),
        # one long prompt chunk after an earlier one: arithmetic
        ("attend_prompt", _cache("attend", 1, 4096, 12000, 32, 8, 128, 128, "bf16")),
        # a few short sessions go back to 16 bits
        ("read_few", _cache("read", 3, 0, 700, 15, 5, 64, 16, "fp16", 19)),
        # every session of a batch does
        ("read_batch", _cache("read", 16, 0, 3000, 32, 32, 128, 64, "bf16", 29)),
        # the text row of one session's tick, its likeliest alternatives
        ("score_one", _score(1, 1, 32000, "f32", 8)),
        # the agent's and user's codebook rows of a full batch, as they lie in the tick's logits
        ("score_audio", _score(64, 16, 2048, "f32", 4, pad=32000)),
        # every position of a few prompts
        ("score_prompt", _score(3001, 1, 32000, "bf16", 20)),
    ]
    return [dict(c, name=n) for n, c in named]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "read", "score"])
    if op == "score":
        n = _spread(rng, 2, 200000)
        inner = rng.choice([1, 1, 2, 16])
        rows = _spread(rng, 1, max(1, min(4000, 90000000 // n // inner)))
        return _score(rows, inner, n, rng.choice(["f32", "f32", "bf16", "fp16"]),
                      rng.choice([0, 1, 5, 20, 64]), rng.random() < 0.7,
                      rng.choice([0, 0, 1, 13, 2048]), rng.choice([0.5, 3.0, 10.0]))
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
        return _cache(op, seqs, chunk, cached, kv_heads * group, kv_heads, dim, page, type, ragged,
                      input=rng.choice([type, type, "f32"]),
                      rot=rng.choice([dim, dim, dim // 2, 2 * rng.randrange(1, dim // 2)]),
                      halves=rng.random() < 0.5, norm=rng.random() < 0.75,
                      far=rng.choice([0, 0, 1000, 2000000]))
    if op == "read":
        seqs = _spread(rng, 1, 32)
        cached = _spread(rng, 1, max(1, min(60000, entries // 4 // seqs)))
        return _cache(op, seqs, 0, cached, kv_heads * group, kv_heads, dim, page, type, ragged)
    seqs = _spread(rng, 1, 64)
    if rng.random() < 0.6:      # single tokens and short chunks, long caches
        chunk = rng.randrange(1, 9)
        cached = _spread(rng, chunk, max(chunk, min(65000, entries // seqs)))
    else:                       # chunks: no more pairs than the largest listed chunk has
        pairs = 4096 * 9000 * 32 // (kv_heads * group)
        cached = _spread(rng, 16, 16000)
        seqs = max(1, min(seqs, entries // cached // 2))
        chunk = _spread(rng, 1, max(1, min(cached, 4096, pairs // cached // seqs)))
    window = rng.choice([0, 0, 0, _spread(rng, 1, cached)])
    return _cache(op, seqs, chunk, cached, kv_heads * group, kv_heads, dim, page, type, ragged,
                  window=window)


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
    if case["op"] == "score":
        rows, size = case["rows"] * case["inner"], 4 if case["type"] == "f32" else 2
        return {"bytes": rows * (case["n"] * size + 8 + 4 * case["entropy"] + 8 * case["top"]),
                "flops": rows * case["n"] * (5 if case["entropy"] else 3)}
    n, total = lengths(case)
    T, H, Hk, D = sum(n), case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        src = 4 if case["input"] == "f32" else 2
        return {"bytes": T * ((H + 2 * Hk) * D * src + H * D * 2 + 2 * Hk * (D + 1) + 4),
                "flops": T * (H + 2 * Hk) * D * 8}
    if case["op"] == "read":
        return {"bytes": sum(total) * Hk * 2 * (D + 1 + 2 * D), "flops": sum(total) * Hk * 2 * D}
    pairs, seen = _visible(case, n, total)
    return {"bytes": 2 * T * H * D * 2 + T * H * 4 + 2 * seen * Hk * (D + 1),
            "flops": 4 * pairs * H * D}


# ---- inputs ------------------------------------------------------------------------------

def _normal(g, *shape, scale=1.0, type=torch.float32):
    out = torch.empty(shape, dtype=type, device=DEVICE)
    return out.normal_(generator=g).mul_(scale)


def _pages(case, per_seq, perm):
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


def _pool(g, *shape):
    """Codes and scales of a pool: normal values of very different size, head by head."""
    x = _normal(g, *shape, type=torch.bfloat16)
    x *= torch.exp2(_normal(g, *shape[:3], 1)).bfloat16()
    return _pack(x)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    if case["op"] == "score":
        return _prepare_score(case, g)
    perm = random.Random(seed)
    n, total = lengths(case)
    T, H, Hk, D, type = sum(n), case["heads"], case["kv_heads"], case["dim"], TYPES[case["type"]]
    cu = [0]
    for c in n:
        cu.append(cu[-1] + c)
    st = {"case": case, "T": T,
          "cu": torch.tensor(cu, dtype=torch.int32, device=DEVICE),
          "len": torch.tensor(total, dtype=torch.int32, device=DEVICE)}
    pool, st["table"] = _pages(case, total, perm)
    shape = (pool, Hk, case["page"], D)
    st["k"], st["k_scale"] = _pool(g, *shape)
    st["v"], st["v_scale"] = _pool(g, *shape)
    # every new token's sequence, entry and place among its sequence's new ones
    st["seq"] = torch.tensor([s for s, c in enumerate(n) for _ in range(c)], dtype=torch.int64,
                             device=DEVICE)
    st["entry"] = torch.tensor([t - c + i for c, t in zip(n, total) for i in range(c)],
                               dtype=torch.int64, device=DEVICE)
    st["nth"] = torch.tensor([i for c in n for i in range(c)], dtype=torch.int64, device=DEVICE)
    if case["op"] == "append":
        src = TYPES[case["input"]]
        # one row holds a token's queries, keys and values, as a joint projection leaves them
        rows = _normal(g, T, (H + 2 * Hk) * D, scale=2.0, type=src)
        st["q_in"], st["k_in"], st["v_in"] = (
            t.unflatten(1, (-1, D)) for t in rows.split([H * D, Hk * D, Hk * D], 1))
        st["q_alpha"] = 1 + _normal(g, D, scale=0.25) if case["norm"] else None
        st["k_alpha"] = 1 + _normal(g, D, scale=0.25) if case["norm"] else None
        st["pos"] = (st["entry"] + case["far"]).int()
    elif case["op"] == "read":
        to, st["to_table"] = _pages(case, total, perm)
        for name in "kv":
            st["to_" + name] = torch.zeros((to,) + shape[1:], dtype=type, device=DEVICE)
    else:
        st["q"] = _normal(g, T, H, D, type=type)
    if own:
        _handles(st)
    return st


def _prepare_score(case, g):
    rows, inner, n = case["rows"], case["inner"], case["n"]
    # rows lie in groups of `inner`, with other logits in front of each group
    all_ = _normal(g, rows, case["pad"] + inner * n, scale=case["spread"], type=TYPES[case["type"]])
    x = all_[:, case["pad"]:].unflatten(1, (inner, n))
    # tokens that the model finds likely, as in earnest: drawn from the rows themselves
    noise = torch.rand(rows, inner, n, generator=g, device=DEVICE).clamp_(min=1e-30)
    tokens = (x.float() - noise.log_().neg_().log_()).argmax(-1).int()
    none = torch.rand(rows, inner, generator=g, device=DEVICE) < 0.05
    tokens[none] = -1                                      # padding
    return {"case": case, "x": x, "tokens": tokens}


# ---- the plain form ------------------------------------------------------------------------

def _pack(y):
    """Codes (e4m3) and scales (the byte e + 127, as e8m0) of each row."""
    y = y.float()
    top = y.abs().amax(-1)
    m, e = torch.frexp(top)                                # top = m 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127)
    e = torch.where(top > 0, e, -127)
    half = torch.div(e, 2, rounding_mode="floor")          # 2^-e by halves: within range
    codes = torch.ldexp(torch.ldexp(y, -half.unsqueeze(-1)), (half - e).unsqueeze(-1)).to(E4M3)
    return codes, (e + 127).to(torch.uint8).view(E8M0)


def _unpack(codes, scale):
    return codes.float() * scale.float().unsqueeze(-1)


def _entries(st, name):
    """All sequences' entries, padded: [seqs, kv_heads, longest, dim], in 32 bits."""
    pages = st["table"].long().clamp(min=0)
    x = _unpack(st[name][pages], st[name + "_scale"][pages])   # [seqs, width, heads, page, dim]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(st):
    case, type = st["case"], st["q"].dtype
    B, C, Hk = case["seqs"], case["chunk"], case["kv_heads"]
    H, D, w = case["heads"], case["dim"], case["window"]
    q = torch.zeros(B, C, H, D, device=DEVICE)
    q[st["seq"], st["nth"]] = st["q"].float()
    at = torch.full((B, C), -1, dtype=torch.int64, device=DEVICE)
    at[st["seq"], st["nth"]] = st["entry"]
    k = _entries(st, "k")
    j = torch.arange(k.shape[2], device=DEVICE)
    hide = j > at.unsqueeze(-1)
    if w:
        hide |= j <= at.unsqueeze(-1) - w
    q = q.unflatten(2, (Hk, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)       # [B, Hk, G C, D]
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5)
    del k
    x = x.unflatten(2, (-1, C)).masked_fill_(hide[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = x.sub_(top).exp_()
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), _entries(st, "v")).unflatten(2, (-1, C)).div_(l)
    lse = (top + l.log()).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[st["seq"], st["nth"]]
    lse = lse.permute(0, 3, 1, 2).flatten(2, 3)[st["seq"], st["nth"]]
    return out.to(type), lse


def _plain_turn(st, x, alpha):
    case = st["case"]
    x = x.float()
    if alpha is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * alpha
    half = case["rot"] // 2
    i = torch.arange(half, dtype=torch.float64, device=DEVICE)
    angle = st["pos"].double()[:, None] * 10000.0 ** (-2.0 * i / case["rot"])
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    lo, hi = (i.long(), i.long() + half) if case["halves"] else (2 * i.long(), 2 * i.long() + 1)
    y = x.clone()
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., lo] * s + x[..., hi] * c
    return y


def _plain_append(st):
    case, type = st["case"], TYPES[st["case"]["type"]]
    q = _plain_turn(st, st["q_in"], st["q_alpha"]).to(type)
    page = st["table"].long()[st["seq"], st["entry"] // case["page"]]
    row = st["entry"] % case["page"]
    k = _pack(_plain_turn(st, st["k_in"], st["k_alpha"]))
    v = _pack(st["v_in"])
    byte = torch.uint8
    st["k"].view(byte)[page, :, row] = k[0].view(byte)
    st["k_scale"].view(byte)[page, :, row] = k[1].view(byte)
    st["v"].view(byte)[page, :, row] = v[0].view(byte)
    st["v_scale"].view(byte)[page, :, row] = v[1].view(byte)
    return q, st["k"], st["k_scale"], st["v"], st["v_scale"]


def _plain_read(st):
    live = torch.arange(st["table"].shape[1] * st["case"]["page"], device=DEVICE) < st["len"][:, None]
    seq, j = live.nonzero(as_tuple=True)
    page, row = st["to_table"].long()[seq, j // st["case"]["page"]], j % st["case"]["page"]
    type = st["to_k"].dtype
    st["to_k"][page, :, row] = _entries(st, "k")[seq, :, j].to(type)
    st["to_v"][page, :, row] = _entries(st, "v")[seq, :, j].to(type)
    return st["to_k"], st["to_v"]


def _plain_score(st):
    case, t = st["case"], st["tokens"]
    x = st["x"].float()
    top = x.amax(-1, keepdim=True)
    e = (x - top).exp()
    lse = top + e.sum(-1, keepdim=True).log()
    given = x.gather(-1, t.long().clamp(min=0).unsqueeze(-1))
    out = {"logprob": torch.where(t < 0, 0.0, (given - lse).squeeze(-1))}
    if case["entropy"]:
        lp = x - lse
        out["entropy"] = -(lp.exp() * lp).sum(-1)
    if case["top"]:
        k = min(case["top"], case["n"])
        v, i = torch.sort(x, dim=-1, descending=True, stable=True)
        ids = torch.full(t.shape + (case["top"],), -1, dtype=torch.int32, device=DEVICE)
        lps = torch.full(ids.shape, -math.inf, device=DEVICE)
        ids[..., :k], lps[..., :k] = i[..., :k].int(), v[..., :k] - lse
        out["top_tokens"], out["top_logprobs"] = ids, lps
    return out


# ---- the framework's calls --------------------------------------------------------------------

def _handles(st):
    import full_duplex_speech_lockstep_gb300 as pp
    st["kv"] = pp.PagedKV8(st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"],
                           dtype=TYPES[st["case"]["type"]])
    if st["case"]["op"] == "read":
        st["to"] = pp.PagedKV(st["to_k"], st["to_v"], st["to_table"])


def _own(st):
    import full_duplex_speech_lockstep_gb300 as pp
    case = st["case"]
    if case["op"] == "score":
        return pp.token_logprobs(st["x"], st["tokens"], top=case["top"],
                                 with_entropy=case["entropy"])
    if "kv" not in st:
        _handles(st)
    kv = st["kv"]
    if case["op"] == "append":
        q = kv.append(st["q_in"], st["k_in"], st["v_in"], st["cu"], st["len"],
                      positions=st["pos"], q_alpha=st["q_alpha"], k_alpha=st["k_alpha"],
                      eps=1e-5, rope_base=10000.0, rot_dim=case["rot"], halves=case["halves"])
        return q, st["k"], st["k_scale"], st["v"], st["v_scale"]
    if case["op"] == "attend":
        return kv.attention(st["q"], st["cu"], st["len"], max_q=case["chunk"],
                            window=case["window"], with_lse=True)
    kv.read(st["len"], st["to"])
    return st["to_k"], st["to_v"]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend, "read": _plain_read,
            "score": _plain_score}[state["case"]["op"]](state)


# ---- the definition in 64 bits ------------------------------------------------------------------

def _e4m3(y):
    """64-bit values to the nearest e4m3 (ties to even): steps of an eighth of their binade, of the
    lowest binade, 2^-6, below it."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _quantised(y):
    """Codes and scales of rows in 64 bits."""
    a = y.abs().amax(-1)
    e = torch.ceil(torch.log2(a / 448.0))
    e = torch.where(a * torch.exp2(-e) > 448.0, e + 1, e)      # where the logarithm was rounded
    e = torch.where(a * torch.exp2(1 - e) <= 448.0, e - 1, e)
    e = torch.where(a > 0, e.clamp(min=-127), torch.full_like(a, -127))
    return _e4m3(y * torch.exp2(-e).unsqueeze(-1)), torch.exp2(e)


def _places(st, count, table):
    """(page, row) of the first entries of a sequence, from its row of a table."""
    j = torch.arange(count, device=DEVICE)
    return table[j // st["case"]["page"]].long(), j % st["case"]["page"]


def _value(st, name, page, head, row):
    return st[name][page, head, row].double() * st[name + "_scale"][page, head, row].double()[:, None]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "score":
        x, t = st["x"].double(), st["tokens"].long()
        p = torch.softmax(x, -1)
        lse = torch.logsumexp(x, -1)
        lp = x.gather(-1, t.clamp(min=0).unsqueeze(-1)).squeeze(-1) - lse
        out = {"logprob": lp * (t >= 0)}
        if case["entropy"]:
            out["entropy"] = lse - (p * x).sum(-1)
        if case["top"]:
            k = min(case["top"], case["n"])
            # the k-th value, then its holders in order: the larger first, the lower index first
            i = torch.argsort(-x, dim=-1, stable=True)[..., :k]
            ids = torch.full(t.shape + (case["top"],), -1, dtype=torch.int32, device=DEVICE)
            lps = torch.full(ids.shape, -math.inf, dtype=torch.float64, device=DEVICE)
            ids[..., :k] = i.int()
            lps[..., :k] = x.gather(-1, i) - lse.unsqueeze(-1)
            out["top_tokens"], out["top_logprobs"] = ids, lps
        return out
    Hk, D = case["kv_heads"], case["dim"]
    n, total = lengths(case)
    first = [sum(n[:s]) for s in range(case["seqs"])]
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
        got = [new["q"]]
        for name in "kv":
            codes, scale = st[name].double(), st[name + "_scale"].double()
            c, s = _quantised(new[name])
            for b in range(case["seqs"]):
                page, row = (z[total[b] - n[b]:] for z in _places(st, total[b], st["table"][b]))
                codes[page, :, row] = c[first[b]:first[b] + n[b]]
                scale[page, :, row] = s[first[b]:first[b] + n[b]]
            got += [codes, scale]
        return tuple(got)
    if case["op"] == "read":
        to = [st["to_k"].double(), st["to_v"].double()]
        for b in range(case["seqs"]):
            page, row = _places(st, total[b], st["table"][b])
            to_page, to_row = _places(st, total[b], st["to_table"][b])
            for pool, name in zip(to, "kv"):
                for h in range(Hk):
                    pool[to_page, h, to_row] = _value(st, name, page, h, row)
        return tuple(to)
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device=DEVICE)
    group = case["heads"] // Hk
    for b in range(case["seqs"]):
        if n[b] == 0:
            continue
        rows = slice(first[b], first[b] + n[b])
        page, row = _places(st, total[b], st["table"][b])
        age = (torch.arange(n[b], device=DEVICE) + (total[b] - n[b]))[:, None, None] - torch.arange(
            total[b], device=DEVICE)
        hidden = (age < 0) | (age >= (case["window"] or total[b] + 1))
        for h in range(Hk):
            heads = slice(h * group, (h + 1) * group)
            k, v = (_value(st, name, page, h, row) for name in "kv")
            x = torch.einsum("igd,jd->igj", st["q"][rows, heads].double(), k) / math.sqrt(D)
            x = x.masked_fill_(hidden, -math.inf)
            lse[rows, heads] = torch.logsumexp(x, -1)
            out[rows, heads] = torch.einsum("igj,jd->igd", torch.softmax(x, -1), v)
    return out, lse
