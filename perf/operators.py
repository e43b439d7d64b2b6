"""Measured cases of the decode-cache operators: rotary positions, appending to a paged
cache, attention over a shared prefix and each sequence's own tokens, selection of the
slots to keep by accumulated attention weight, and the eviction itself.

``run`` computes an operator in plain torch (32-bit arithmetic, angles in 64 bits, one
rounding at the end) while ``own`` is false, and through the package's public calls while
it is true.  ``exact`` evaluates the same definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------ cases --
def listed():
    return [
        # one long prompt: the 16 query heads of a 32768-token prefill, halves layout
        {"name": "rope_prefill", "op": "rope", "n_tok": 32768, "heads": 16, "d": 128, "rot_begin": 0, "rot": 128,
         "inter": False, "inverse": False, "dtype": "bf16", "pos0": 0, "base": 1e6, "factor": 4.0},
        # gradient of index queries whose last 32 of 64 dimensions rotate, pairs interleaved,
        # far into a long document
        {"name": "rope_index_grad", "op": "rope", "n_tok": 8191, "heads": 4, "d": 64, "rot_begin": 32, "rot": 32,
         "inter": True, "inverse": True, "dtype": "f32", "pos0": 1000000, "base": 1e4, "factor": 1.0},
        # a decode step's new token of 64 sequences: queries rotated, keys and values stored
        {"name": "append_step", "op": "append", "n_seq": 64, "n_tok": 1, "n_q": 32, "n_kv": 8, "d": 128, "rot": 128,
         "inter": False, "page": 64, "own_min": 1, "own_max": 1024, "ragged": False, "prefix": 32768},
        # chunks of prompts of different lengths, padded to the longest
        {"name": "append_chunk", "op": "append", "n_seq": 12, "n_tok": 1000, "n_q": 32, "n_kv": 8, "d": 128,
         "rot": 64, "inter": True, "page": 16, "own_min": 0, "own_max": 100, "ragged": True, "prefix": 777},
        # one user right after a short system prompt: latency
        {"name": "attn_one", "op": "attn", "n_seq": 1, "n_tok": 1, "n_q": 16, "n_kv": 1, "d": 128, "prefix": 1000,
         "own_min": 37, "own_max": 37, "page": 64, "out": "bf16", "mass": False, "ragged": False},
        # 64 sequences on one 32768-token document, weights accumulated for eviction
        {"name": "attn_batch", "op": "attn", "n_seq": 64, "n_tok": 1, "n_q": 32, "n_kv": 8, "d": 128,
         "prefix": 32768, "own_min": 1, "own_max": 2047, "page": 64, "out": "bf16", "mass": True, "ragged": False},
        # many samples from one long prompt: the shared part is a large matrix product
        {"name": "attn_wide", "op": "attn", "n_seq": 256, "n_tok": 1, "n_q": 32, "n_kv": 4, "d": 128,
         "prefix": 16384, "own_min": 0, "own_max": 511, "page": 64, "out": "bf16", "mass": False, "ragged": False},
        # up to five drafted tokens checked per sequence, some sequences idle, odd sizes, 32-bit outputs
        {"name": "attn_draft", "op": "attn", "n_seq": 23, "n_tok": 5, "n_q": 24, "n_kv": 8, "d": 64, "prefix": 5001,
         "own_min": 0, "own_max": 333, "page": 24, "out": "f32", "mass": True, "ragged": True},
        # the per-step choice of half of a 2048-slot budget
        {"name": "select_step", "op": "select", "n_seq": 64, "n_kv": 8, "len_min": 1024, "len_max": 2048,
         "keep": 1024, "sink": 4, "window": 64},
        # a long document cut to 4096 slots per head
        {"name": "select_long", "op": "select", "n_seq": 32, "n_kv": 4, "len_min": 30000, "len_max": 32768,
         "keep": 4096, "sink": 4, "window": 512},
        # a small cache trimmed often
        {"name": "evict_step", "op": "evict", "n_seq": 8, "n_kv": 8, "d": 128, "page": 16, "len_min": 700,
         "len_max": 1100, "keep": 768},
        # the long caches' rows moved into the freed slots
        {"name": "evict_long", "op": "evict", "n_seq": 16, "n_kv": 8, "d": 128, "page": 64, "len_min": 8000,
         "len_max": 16384, "keep": 4096},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _largest(op):
    w = [work(c) for c in listed() if c["op"] == op]
    return max(x["bytes"] for x in w), max(x["flops"] for x in w)


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "select", "evict"])
    most_bytes, most_flops = _largest(op)
    while True:
        c = _draw_one(rng, op)
        w = work(c)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return c


def _draw_one(rng, op):
    d = rng.choice([64, 128, 128])
    n_q, n_kv = rng.choice([(16, 1), (32, 8), (32, 4), (24, 8), (8, 8), (14, 2), (64, 4)])
    page = rng.choice([16, 24, 32, 64, 100, 128])
    if op == "rope":
        rot = rng.choice([d, d, d // 2, 20])
        return {"op": op, "n_tok": _log(rng, 1, 32768), "heads": rng.choice([1, 3, 4, 8, 16, 40]), "d": d,
                "rot_begin": rng.choice([0, d - rot]), "rot": rot, "inter": rng.random() < 0.5,
                "inverse": rng.random() < 0.4, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "pos0": rng.choice([0, 4095, 131072, 2000000]), "base": rng.choice([1e4, 5e5, 1e6]),
                "factor": rng.choice([1.0, 4.0, 32.0])}
    if op == "append":
        lo = rng.choice([0, 1, 50])
        return {"op": op, "n_seq": _log(rng, 1, 128), "n_tok": rng.choice([1, 1, _log(rng, 2, 1000)]), "n_q": n_q,
                "n_kv": n_kv, "d": d, "rot": rng.choice([d, d // 2]), "inter": rng.random() < 0.5, "page": page,
                "own_min": lo, "own_max": lo + _log(rng, 1, 1000), "ragged": rng.random() < 0.5,
                "prefix": rng.choice([0, 1000, 131072])}
    if op == "attn":
        lo = rng.choice([0, 1, 100])
        return {"op": op, "n_seq": _log(rng, 1, 256), "n_tok": rng.choice([1, 1, 1, 2, 3, 5, 8]), "n_q": n_q,
                "n_kv": n_kv, "d": d, "prefix": rng.choice([0, _log(rng, 1, 32768), _log(rng, 256, 32768)]),
                "own_min": lo, "own_max": lo + _log(rng, 1, 4096), "page": page,
                "out": rng.choice(["bf16", "bf16", "f32"]), "mass": rng.random() < 0.5, "ragged": rng.random() < 0.3}
    if op == "select":
        hi = _log(rng, 64, 32768)
        return {"op": op, "n_seq": _log(rng, 1, 64), "n_kv": rng.choice([1, 4, 8]), "len_min": max(1, hi // 3),
                "len_max": hi, "keep": max(32, int(hi * rng.uniform(0.1, 0.9))), "sink": rng.choice([0, 4]),
                "window": rng.choice([0, 1, 16])}
    hi = _log(rng, 64, 16384)
    return {"op": op, "n_seq": _log(rng, 1, 64), "n_kv": rng.choice([1, 4, 8]), "d": d, "page": page,
            "len_min": max(1, hi // 2), "len_max": hi, "keep": max(1, int(hi * rng.uniform(0.1, 0.9)))}


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    if n == 1:
        return [hi]
    return [lo + ((hi - lo) * i) // (n - 1) for i in range(n)]


def _new(case):
    """New tokens of each sequence: all of them, or 0 .. n_tok."""
    return _spread(0 if case["n_seq"] > 1 else 1, case["n_tok"], case["n_seq"]) if case["ragged"] else \
        [case["n_tok"]] * case["n_seq"]


def work(case):
    """Each input read once, each output written once."""
    op = case["op"]
    if op == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["n_tok"] * case["heads"]
        return {"bytes": 2 * n * case["d"] * size + 4 * case["n_tok"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    if op == "append":
        rows = sum(_new(case))
        heads = case["n_q"] + 2 * case["n_kv"]
        return {"bytes": rows * (2 * heads * case["d"] * 2 + 8 * case["n_kv"]) + 16 * case["n_seq"],
                "flops": 3 * rows * (case["n_q"] + case["n_kv"]) * case["rot"]}
    if op == "attn":
        own_len = _spread(case["own_min"], case["own_max"], case["n_seq"])
        # the sequences' lengths and their new tokens are paired at random: count the mean
        new = _new(case)
        held, asked = sum(own_len) + sum(new), sum(new)
        pairs = asked * case["prefix"] + asked * sum(own_len) / case["n_seq"] + sum(n * (n + 1) // 2 for n in new)
        rows = case["n_seq"] * case["n_tok"] * case["n_q"]
        b = (case["prefix"] + held) * case["n_kv"] * case["d"] * 4
        b += rows * (case["d"] * (2 + (2 if case["out"] == "bf16" else 4)) + 4)
        b += held * case["n_kv"] * 8 if case["mass"] else 0
        return {"bytes": b, "flops": 4 * case["d"] * case["n_q"] * pairs}
    lens = _spread(case["len_min"], case["len_max"], case["n_seq"])
    rows = case["n_seq"] * case["n_kv"]
    if op == "select":
        return {"bytes": sum(lens) * case["n_kv"] * 8 + rows * case["keep"] * 4, "flops": sum(lens) * case["n_kv"]}
    # evict: a row moves when it is kept and stands past the budget; kept slots are spread evenly
    moved = sum(case["keep"] * (1.0 - case["keep"] / n) for n in lens if n > case["keep"]) * case["n_kv"]
    return {"bytes": moved * (8 * case["d"] + 16) + rows * case["keep"] * 4, "flops": moved}


# ----------------------------------------------------------------------------- inputs --
def _inv_freq(rot, base, factor):
    """Radians per position of each pair, stretched by `factor` for contexts past the trained one."""
    j = torch.arange(0, rot, 2, dtype=torch.float64, device=DEV)
    return base ** (-j / rot) / factor


def _permuted(values, gen, dtype=torch.int32):
    order = torch.randperm(len(values), generator=gen, device=DEV)
    return torch.tensor(values, dtype=dtype, device=DEV)[order]


def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _pools(st, gen, n_seq, n_kv, d, page, slots):
    """A page pool in which the sequences' pages interleave, and their block table."""
    max_pages = -(-slots // page)
    n_pages = n_seq * max_pages
    st["cap"] = max_pages * page
    st["block_table"] = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32).view(n_seq, max_pages)
    st["k_pool"] = _randn(gen, n_pages, page, n_kv, d)
    st["v_pool"] = _randn(gen, n_pages, page, n_kv, d)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    st = {"op": case["op"], "case": case}
    if case["op"] == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["x"] = _randn(gen, case["n_tok"], case["heads"], case["d"], dtype=dt)
        st["pos"] = torch.arange(case["pos0"], case["pos0"] + case["n_tok"], dtype=torch.int32, device=DEV)
        st["inv_freq"] = _inv_freq(case["rot"], case["base"], case["factor"])
        st["mscale"] = 0.1 * math.log(case["factor"]) + 1.0
        return st
    n_seq, n_kv = case["n_seq"], case["n_kv"]
    if case["op"] in ("append", "attn"):
        n_tok, n_q, d = case["n_tok"], case["n_q"], case["d"]
        _pools(st, gen, n_seq, n_kv, d, case["page"], case["own_max"] + n_tok)
        st["seq_len"] = _permuted(_spread(case["own_min"], case["own_max"], n_seq), gen)
        st["n_new"] = _permuted(_new(case), gen) if case["ragged"] else None
        st["next_pos"] = st["seq_len"] + case["prefix"]
        st["pos"] = (torch.arange(st["cap"], dtype=torch.int32, device=DEV) + case["prefix"]).repeat(n_seq, n_kv, 1)
        st["q"] = _randn(gen, n_seq, n_tok, n_q, d)
        if case["op"] == "append":
            st["k"] = _randn(gen, n_seq, n_tok, n_kv, d)
            st["v"] = _randn(gen, n_seq, n_tok, n_kv, d)
            st["inv_freq"] = _inv_freq(case["rot"], 1e6, 1.0)
            st["mass"] = torch.rand(n_seq, n_kv, st["cap"], generator=gen, device=DEV)
        else:
            st["prefix_k"] = _randn(gen, case["prefix"], n_kv, d)
            st["prefix_v"] = _randn(gen, case["prefix"], n_kv, d)
            st["mass"] = torch.rand(n_seq, n_kv, st["cap"], generator=gen, device=DEV) if case["mass"] else None
            st["mass_out"] = st["mass"].clone() if case["mass"] else None
    else:
        lens = _permuted(_spread(case["len_min"], case["len_max"], n_seq), gen)
        st["seq_len"], st["next_pos"], st["keep"] = lens, lens.clone(), case["keep"]
        page = case.get("page", 1)
        cap = -(-case["len_max"] // page) * page
        # heavy-tailed weights; tokens that no query has looked at yet stay at zero
        mass = torch.rand(n_seq, n_kv, cap, generator=gen, device=DEV).pow_(8)
        mass[torch.rand(n_seq, n_kv, cap, generator=gen, device=DEV) < 0.05] = 0.0
        st["mass"] = mass
        st["pos"] = torch.arange(cap, dtype=torch.int32, device=DEV).repeat(n_seq, n_kv, 1)
        if case["op"] == "evict":
            _pools(st, gen, n_seq, n_kv, case["d"], page, cap)
            st["idx"], st["count"] = _plain_select(mass, lens, lens, st["pos"], case["keep"], 0, 0)
    if own and case["op"] != "select":
        import content_routed_sparse_b200 as crs
        st["cache"] = crs.KvCache(st["k_pool"], st["v_pool"], st["block_table"], st["seq_len"], st["next_pos"],
                                  pos=st["pos"], mass=st["mass"])
    return st


# ------------------------------------------------------------------------------- runs --
def run(state):
    op = state["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attn": _own_attn, "select": _own_select,
                "evict": _own_evict}[op](state)
    return {"rope": _run_rope, "append": _run_append, "attn": _run_attn, "select": _run_select,
            "evict": _run_evict}[op](state)


def _own_rope(st):
    import content_routed_sparse_b200 as crs
    c = st["case"]
    return crs.rope(st["x"], st["pos"], st["inv_freq"], rot_begin=c["rot_begin"], interleaved=c["inter"],
                    mscale=st["mscale"], inverse=c["inverse"])


def _own_append(st):
    q = st["cache"].append(st["k"], st["v"], q=st["q"], inv_freq=st["inv_freq"], n_new=st["n_new"],
                           interleaved=st["case"]["inter"])
    return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"], "pos": st["pos"], "mass": st["mass"]}


def _own_attn(st):
    dt = torch.bfloat16 if st["case"]["out"] == "bf16" else torch.float32
    o, lse = st["cache"].attend(st["q"], st["prefix_k"], st["prefix_v"], n_new=st["n_new"], out_dtype=dt,
                                mass_out=st["mass_out"])
    return {"o": o, "lse": lse, "mass": st["mass_out"]}


def _own_select(st):
    import content_routed_sparse_b200 as crs
    c = st["case"]
    idx, count = crs.mass_select(st["mass"], st["seq_len"], c["keep"], pos=st["pos"], next_pos=st["next_pos"],
                                 sink_end=c["sink"], window=c["window"])
    return {"idx": idx, "count": count}


def _own_evict(st):
    st["cache"].evict(st["idx"], st["count"])
    return {"k_pool": st["k_pool"], "v_pool": st["v_pool"], "mass": st["mass"], "pos": st["pos"],
            "seq_len": st["seq_len"]}


# ------------------------------------------------------------------------ plain forms --
def _rotate(x, pos, inv_freq, rot_begin, inter, mscale, inverse):
    """x [..., heads, d] at positions pos [...]; angles in 64 bits, the rotation in 32."""
    rot = 2 * inv_freq.numel()
    ang = pos.double()[..., None, None] * inv_freq
    cos, sin = (ang.cos() * mscale).float(), (ang.sin() * (-mscale if inverse else mscale)).float()
    y = x.float().clone()
    part = y[..., rot_begin:rot_begin + rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if inter else (part[..., :rot // 2], part[..., rot // 2:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    a.copy_(ra)
    b.copy_(rb)
    return y.to(x.dtype)


def _run_rope(st):
    c = st["case"]
    return _rotate(st["x"], st["pos"], st["inv_freq"], c["rot_begin"], c["inter"], st["mscale"], c["inverse"])


def _live(st, n_tok):
    """[n_seq, n_tok]: which of the padded new tokens exist."""
    n_seq = st["seq_len"].numel()
    if st["n_new"] is None:
        return torch.ones(n_seq, n_tok, dtype=torch.bool, device=DEV)
    return torch.arange(n_tok, device=DEV)[None, :] < st["n_new"][:, None]


def _run_append(st):
    c = st["case"]
    n_tok, page = c["n_tok"], c["page"]
    live = _live(st, n_tok)
    i = torch.arange(n_tok, device=DEV)
    at = st["next_pos"][:, None] + i
    q = _rotate(st["q"], at, st["inv_freq"], 0, c["inter"], 1.0, False)
    q = torch.where(live[..., None, None], q, torch.zeros_like(q))
    k = _rotate(st["k"], at, st["inv_freq"], 0, c["inter"], 1.0, False)
    s, t = live.nonzero(as_tuple=True)
    slot = (st["seq_len"][:, None] + i)[s, t].long()
    where = st["block_table"][s, slot // page].long()
    st["k_pool"][where, slot % page] = k[s, t]
    st["v_pool"][where, slot % page] = st["v"][s, t]
    st["pos"][s, :, slot] = at[s, t].to(torch.int32)[:, None]
    st["mass"][s, :, slot] = 0.0
    return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"], "pos": st["pos"], "mass": st["mass"]}


def _run_attn(st):
    c = st["case"]
    n_seq, n_tok, n_q, n_kv, d = c["n_seq"], c["n_tok"], c["n_q"], c["n_kv"], c["d"]
    g, cap, tp = n_q // n_kv, st["cap"], c["prefix"]
    live = _live(st, n_tok)
    new = live.sum(1)
    total = st["seq_len"] + new
    q = st["q"].float().view(n_seq, n_tok, n_kv, g, d).permute(2, 0, 1, 3, 4)          # [kv, seq, tok, g, d]
    scale = 1.0 / math.sqrt(d)
    pk, pv = st["prefix_k"].float().permute(1, 0, 2), st["prefix_v"].float().permute(1, 0, 2)
    sp = torch.matmul(q.reshape(n_kv, n_seq * n_tok * g, d), pk.transpose(1, 2)).view(n_kv, n_seq, n_tok, g, tp)
    table = st["block_table"].long()
    ok = st["k_pool"][table].view(n_seq, cap, n_kv, d).permute(2, 0, 1, 3).float()     # [kv, seq, cap, d]
    ov = st["v_pool"][table].view(n_seq, cap, n_kv, d).permute(2, 0, 1, 3).float()
    so = torch.matmul(q.reshape(n_kv, n_seq, n_tok * g, d), ok.transpose(2, 3)).view(n_kv, n_seq, n_tok, g, cap)
    # token i of the new ones sees the slots before its own and itself
    last = (total - new)[:, None] + torch.arange(n_tok, device=DEV)
    seen = (torch.arange(cap, device=DEV) <= last[..., None]) & live[..., None]
    so = so.masked_fill(~seen[None, :, :, None, :], -math.inf)
    sp = sp.masked_fill(~live[None, :, :, None, None], -math.inf)
    s = torch.cat([sp, so], -1).mul_(scale)
    m = s.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    lse = m + torch.log(z)
    p = p / z.masked_fill(z == 0, 1.0)
    o = torch.matmul(p[..., :tp].reshape(n_kv, n_seq * n_tok * g, tp), pv).view(n_kv, n_seq, n_tok, g, d)
    o = o + torch.matmul(p[..., tp:].reshape(n_kv, n_seq, n_tok * g, cap), ov).view(n_kv, n_seq, n_tok, g, d)
    o = o.permute(1, 2, 0, 3, 4).reshape(n_seq, n_tok, n_q, d)
    o = o.to(torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    lse = lse[..., 0].permute(1, 2, 0, 3).reshape(n_seq, n_tok, n_q)
    mass = None
    if st["mass"] is not None:
        held = torch.arange(cap, device=DEV) < total[:, None]
        mass = st["mass"] + p[..., tp:].sum((2, 3)).permute(1, 0, 2) * held[:, None, :]
    return {"o": o, "lse": lse, "mass": mass}


def _plain_select(mass, seq_len, next_pos, pos, keep, sink, window):
    n_seq, n_kv, cap = mass.shape
    slot = torch.arange(cap, device=DEV)
    held = (slot < seq_len[:, None])[:, None, :]
    fixed = (pos < sink) | (pos >= (next_pos - window)[:, None, None])
    score = mass.masked_fill(fixed, math.inf).masked_fill(~held, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    count = seq_len.clamp(max=keep)
    rank = torch.arange(order.shape[-1], device=DEV)
    order = torch.where(rank < count[:, None, None], order, cap + 1)
    idx = torch.sort(order, dim=-1).values
    idx = torch.where(idx > cap, -1, idx).to(torch.int32)
    if idx.shape[-1] < keep:
        idx = torch.nn.functional.pad(idx, (0, keep - idx.shape[-1]), value=-1)
    return idx.contiguous(), count.to(torch.int32)


def _run_select(st):
    c = st["case"]
    idx, count = _plain_select(st["mass"], st["seq_len"], st["next_pos"], st["pos"], c["keep"], c["sink"],
                               c["window"])
    return {"idx": idx, "count": count}


def _run_evict(st):
    """The r-th kept slot at or past the new length moves to the r-th free slot before it."""
    c, idx, count = st["case"], st["idx"].long(), st["count"].long()
    keep, cap, page = c["keep"], st["mass"].shape[-1], c["page"]
    lim = count[:, None, None]
    kept = torch.zeros(idx.shape[0], idx.shape[1], cap + 1, dtype=torch.bool, device=DEV)
    kept.scatter_(2, torch.where(idx < 0, cap, idx), True)
    slot = torch.arange(cap, device=DEV)
    hole = ~kept[..., :cap] & (slot < lim)
    source = kept[..., :cap] & (slot >= lim)
    s, h, dst = hole.nonzero(as_tuple=True)           # rows and slots ascending in both lists
    _, _, src = source.nonzero(as_tuple=True)
    table = st["block_table"].long()
    sp, dp = table[s, src // page], table[s, dst // page]
    for pool in (st["k_pool"], st["v_pool"]):
        pool[dp, dst % page, h] = pool[sp, src % page, h]
    for meta in (st["mass"], st["pos"]):
        meta[s, h, dst] = meta[s, h, src]
    st["seq_len"].copy_(count)
    return {"k_pool": st["k_pool"], "v_pool": st["v_pool"], "mass": st["mass"], "pos": st["pos"],
            "seq_len": st["seq_len"]}


# --------------------------------------------------------------------------- 64 bits --
def _exact_turn(x, pos, inv_freq, rot_begin, inter, mscale, sign):
    """Rotation by complex multiplication: (a + ib) e^{i pos w}."""
    half = inv_freq.numel()
    out = x.double().clone()
    j = torch.arange(half, device=DEV)
    ia, ib = (rot_begin + 2 * j, rot_begin + 2 * j + 1) if inter else (rot_begin + j, rot_begin + half + j)
    z = torch.complex(out[..., ia], out[..., ib])
    w = torch.polar(torch.full((), mscale, dtype=torch.float64, device=DEV),
                    sign * pos.double()[..., None, None] * inv_freq)
    z = z * w
    out[..., ia] = z.real
    out[..., ib] = z.imag
    return out


def exact(case, seed):
    if case["op"] in ("select", "evict"):
        return None                       # whole numbers and copied rows
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(st["x"], st["pos"], st["inv_freq"], case["rot_begin"], case["inter"], st["mscale"],
                           -1.0 if case["inverse"] else 1.0)
    new = [case["n_tok"]] * case["n_seq"] if st["n_new"] is None else st["n_new"].tolist()
    lens = st["seq_len"].tolist()
    if case["op"] == "append":
        q = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
        k = st["k_pool"].double()
        for s, n in enumerate(new):
            at = st["next_pos"][s] + torch.arange(n, device=DEV)
            q[s, :n] = _exact_turn(st["q"][s, :n], at, st["inv_freq"], 0, case["inter"], 1.0, 1.0)
            slot = lens[s] + torch.arange(n, device=DEV)
            k[st["block_table"][s, slot // case["page"]].long(), slot % case["page"]] = \
                _exact_turn(st["k"][s, :n], at, st["inv_freq"], 0, case["inter"], 1.0, 1.0)
        return {"q": q, "k_pool": k, "v_pool": None, "pos": None, "mass": None}
    n_tok, n_q, n_kv, d = case["n_tok"], case["n_q"], case["n_kv"], case["d"]
    g = n_q // n_kv
    o = torch.zeros(case["n_seq"], n_tok, n_q, d, dtype=torch.float64, device=DEV)
    lse = torch.full((case["n_seq"], n_tok, n_q), -math.inf, dtype=torch.float64, device=DEV)
    mass = st["mass"].double() if case["mass"] else None
    pk = st["prefix_k"].double().permute(1, 2, 0).contiguous()                         # [kv, d, prefix]
    pv = st["prefix_v"].double().permute(1, 0, 2).contiguous()
    for s, n in enumerate(new):
        if n == 0:
            continue
        t = lens[s] + n
        pages = st["block_table"][s].long()
        ks = st["k_pool"][pages].reshape(-1, n_kv, d)[:t].double().permute(1, 2, 0)
        vs = st["v_pool"][pages].reshape(-1, n_kv, d)[:t].double().permute(1, 0, 2)
        qs = st["q"][s, :n].double().view(n, n_kv, g, d).permute(1, 0, 2, 3).reshape(n_kv, n * g, d) / math.sqrt(d)
        far = torch.bmm(qs, pk)
        near = torch.bmm(qs, ks).view(n_kv, n, g, t)
        hidden = torch.arange(t, device=DEV)[None, :] > (lens[s] + torch.arange(n, device=DEV))[:, None]
        near = near.masked_fill(hidden[None, :, None, :], -math.inf).view(n_kv, n * g, t)
        z = torch.logaddexp(torch.logsumexp(near, -1), torch.logsumexp(far, -1)) if case["prefix"] else \
            torch.logsumexp(near, -1)
        wn = (near - z[..., None]).exp()
        os_ = torch.bmm(wn, vs) + torch.bmm((far - z[..., None]).exp(), pv)
        o[s, :n] = os_.view(n_kv, n, g, d).permute(1, 0, 2, 3).reshape(n, n_q, d)
        lse[s, :n] = z.view(n_kv, n, g).permute(1, 0, 2).reshape(n, n_q)
        if mass is not None:
            mass[s, :, :t] += wn.sum(1)
    return {"o": o, "lse": lse, "mass": mass}
