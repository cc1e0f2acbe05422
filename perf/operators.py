"""The operators between the QKV product and the output projection, measured.

Kinds of cases:
  rope   - RMSNorm of every query and key head and the rotation by position, one pass;
  append - a step's keys and values quantised into the paged 4-bit cache, and read back;
  plan   - page tables, slots and positions of a step from the requests' lengths;
  attn   - causal attention of a step's queries over the paged 4-bit cache.

Cache layout (one pool each for keys and values): codes int32 [pages, heads, page, D/8],
scale and zero f32 [pages, heads, page, D/gs, 2], value = (code - zero) * scale.  With J = D/32
and u = d/32: code d of a key row is nibble d%8 of word ((d%32)/8)*J + u; of a value row it is
nibble d%4 of the 16-bit half ((d%32)/4)*J + u (halves counted from the low one up).
"""

import math

import torch

own = False


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _case(name, kind, **kw):
    return {"name": name, "kind": kind, **kw}


def listed():
    return [
        # one decoding request: latency of the smallest call
        _case("rope_one", "rope", tokens=1, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False,
              norm=True, fused=False),
        # a prompt whose q and k are columns of one fused projection, half of each head rotated
        _case("rope_prompt", "rope", tokens=8191, heads=32, kv_heads=8, dim=128, rot=64, interleaved=True,
              norm=True, fused=True),
        # one decode step of 61 requests
        _case("append_step", "append", tokens=61, kv_heads=8, dim=128, group=64, page=16),
        # a long prompt
        _case("append_prompt", "append", tokens=16381, kv_heads=8, dim=128, group=128, page=64),
        # a decode step of 64 requests, one new token each
        _case("plan_step", "plan", requests=64, new_most=1, past_most=4096, page=16),
        # many prompts at once
        _case("plan_prompts", "plan", requests=2000, new_most=256, past_most=2048, page=16),
        # one request, a short context: latency
        _case("attn_one", "attn", requests=1, new=1, past_least=776, past_most=776, heads=32, kv_heads=8,
              dim=128, group=128, page=16, window=0),
        # the ordinary decode step: a ragged batch
        _case("attn_batch", "attn", requests=48, new=1, past_least=500, past_most=8192, heads=32, kv_heads=8,
              dim=128, group=128, page=16, window=0),
        # two long documents, finer groups
        _case("attn_long", "attn", requests=2, new=1, past_least=120000, past_most=131071, heads=32, kv_heads=8,
              dim=128, group=64, page=64, window=0),
        # drafted tokens checked together; a head for each query, the finest groups
        _case("attn_draft", "attn", requests=16, new=5, past_least=100, past_most=4096, heads=16, kv_heads=16,
              dim=64, group=32, page=32, window=0),
        # chunks of prompts after earlier chunks, with a sliding window
        _case("attn_chunk", "attn", requests=3, new=1021, past_least=1000, past_most=4096, heads=32, kv_heads=8,
              dim=128, group=32, page=16, window=2048),
        # a whole prompt
        _case("attn_prompt", "attn", requests=1, new=6007, past_least=0, past_most=0, heads=32, kv_heads=8,
              dim=128, group=128, page=64, window=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "plan", "attn", "attn", "attn"])
    dim = rng.choice([64, 96, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 5, 8])
    ratio = rng.choice([1, 2, 4, 5, 7, 8])
    group = rng.choice([g for g in (32, 64, 96, 128, 256) if dim % g == 0])
    page = rng.choice([16, 32, 64, 128])
    if kind == "rope":
        most = 8191 * 40 * 128 // ((ratio + 1) * kv * dim)
        return {"kind": kind, "tokens": _log(rng, 1, min(most, 20000)), "heads": ratio * kv, "kv_heads": kv,
                "dim": dim, "rot": rng.choice([dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.5,
                "norm": rng.random() < 0.7, "fused": rng.random() < 0.5}
    if kind == "append":
        most = 16381 * 8 * 128 // (kv * dim)
        return {"kind": kind, "tokens": _log(rng, 1, min(most, 40000)), "kv_heads": kv, "dim": dim,
                "group": group, "page": page}
    if kind == "plan":
        return {"kind": kind, "requests": _log(rng, 1, 2000), "new_most": _log(rng, 1, 256),
                "past_most": _log(rng, 1, 2048), "page": page}
    heads = ratio * kv
    new = 1 if rng.random() < 0.4 else _log(rng, 1, 2000)
    length = _log(rng, 1, 40000)
    # within the listed prompt's products and rows, and the listed caches' bytes
    flops, rows, codes = 4 * 128 * 32 * 6007 * 3004, 128 * 32 * 6007, 131072 * 2 * 8 * 128
    new = max(1, min(new, rows // (heads * dim)))
    length = max(1, min(length, flops // (4 * heads * dim * new) - new // 2, codes // (kv * dim) - new))
    most = min(flops // (4 * heads * dim * new * (length + new // 2 + 1)), rows // (heads * dim * new),
               codes // (kv * dim * (length + new)))
    most = max(1, most)
    return {"kind": kind, "requests": _log(rng, 1, min(64, most)), "new": new, "past_least": rng.choice([0, length // 2]),
            "past_most": length, "heads": heads, "kv_heads": kv, "dim": dim, "group": group, "page": page,
            "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0x6751 + int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(g, lo, hi, *shape):
    """Whole numbers of lo..hi, both ends among them."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _lengths(case, seed):
    """The requests' past lengths of an attention case, on the host (work() needs them too)."""
    g = torch.Generator()
    g.manual_seed(0x51 + int(seed))
    return torch.randint(case["past_least"], case["past_most"] + 1, (case["requests"],), generator=g)


def _channels(g, heads, dim):
    """Keys and values have channels of unlike size and offset."""
    return torch.exp(0.3 * _randn(g, heads, dim)), 0.3 * _randn(g, heads, dim)


def _codes(x, group):
    """The quantiser's rule, each step one rounding in 32 bits: codes int32 [..., D], scale and zero [..., D/gs, 2]."""
    v = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    lo = v.amin(-1, keepdim=True) + 0.0
    hi = v.amax(-1, keepdim=True) + 0.0
    s = (hi - lo) / torch.full_like(hi, 15.0)  # a quotient: by a plain number it may become a product
    s = torch.where(s < torch.finfo(torch.float32).tiny, torch.ones_like(s), s)
    q = torch.round((v - lo) * (1.0 / s)).clamp(0, 15).to(torch.int32)
    return q.reshape(x.shape), torch.cat([s, -lo / s], -1)


def _pack_keys(q):
    J = q.shape[-1] // 32
    w = q.reshape(*q.shape[:-1], J, 4, 8).transpose(-3, -2)
    sh = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)
    return (w << sh).sum(-1, dtype=torch.int32).reshape(*q.shape[:-1], 4 * J)


def _pack_values(q):
    J = q.shape[-1] // 32
    h = q.reshape(*q.shape[:-1], J, 8, 4).transpose(-3, -2).reshape(*q.shape[:-1], 4 * J, 2, 4)
    sh = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32).reshape(2, 4)
    return (h << sh).sum((-2, -1), dtype=torch.int32)


def _unpack_keys(w):
    J = w.shape[-1] // 4
    sh = torch.arange(0, 32, 4, device=w.device, dtype=torch.int32)
    q = (w.unsqueeze(-1) >> sh) & 15
    return q.reshape(*w.shape[:-1], 4, J, 8).transpose(-3, -2).reshape(*w.shape[:-1], 32 * J)


def _unpack_values(w):
    J = w.shape[-1] // 4
    sh = torch.arange(0, 32, 4, device=w.device, dtype=torch.int32)
    q = (w.unsqueeze(-1) >> sh) & 15
    return q.reshape(*w.shape[:-1], 8, J, 4).transpose(-3, -2).reshape(*w.shape[:-1], 32 * J)


def _values(q, sz, dtype=torch.float32):
    """(code - zero) * scale."""
    G = sz.shape[-2]
    v = q.to(dtype).reshape(*q.shape[:-1], G, q.shape[-1] // G)
    sz = sz.to(dtype)
    return ((v - sz[..., 1:]) * sz[..., :1]).reshape(q.shape)


def _prepare_rope(case, seed):
    g = _gen(seed)
    T, H, KH, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    if case["fused"]:  # q, k and v side by side, as one projection leaves them
        qkv = _randn(g, T, H + 2 * KH, D)
        q, k = qkv[:, :H], qkv[:, H:H + KH]
    else:
        q, k = _randn(g, T, H, D), _randn(g, T, KH, D)
    half = case["rot"] // 2
    inv = (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
    start = int(_ints(g, 0, 200000, 1)[0])
    return {"case": case, "q": q, "k": k, "inv": inv,
            "positions": (start + torch.arange(T, device="cuda")).to(torch.int32),
            "q_gain": 1.0 + 0.2 * _randn(g, D) if case["norm"] else None,
            "k_gain": 1.0 + 0.2 * _randn(g, D) if case["norm"] else None}


def _pool(pages, kv_heads, page, dim, group):
    words = torch.zeros(pages, kv_heads, page, dim // 8, dtype=torch.int32, device="cuda")
    sz = torch.zeros(pages, kv_heads, page, dim // group, 2, device="cuda")
    return words, sz


def _prepare_append(case, seed):
    g = _gen(seed)
    T, KH, D, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    gain, mid = _channels(g, KH, D)
    k = _randn(g, T, KH, D) * gain + mid
    v = _randn(g, T, KH, D)
    pages = (T + page - 1) // page + 7
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    t = torch.arange(T, device="cuda")
    slots = (order[t // page] * page + t % page).to(torch.int32)
    kq, ksz = _pool(pages, KH, page, D, case["group"])
    vq, vsz = _pool(pages, KH, page, D, case["group"])
    return {"case": case, "k": k, "v": v, "slots": slots, "kq": kq, "ksz": ksz, "vq": vq, "vsz": vsz}


def _prepare_plan(case, seed):
    g = _gen(seed)
    B, page = case["requests"], case["page"]
    past = _ints(g, 0, case["past_most"], B)
    new = _ints(g, 1, case["new_most"], B)
    most = (case["past_most"] + case["new_most"] + page - 1) // page
    had = (past + page - 1) // page
    need = (past + new + page - 1) // page - had
    total, granted = int(had.sum()), int(need.sum())
    order = torch.randperm(total + granted + 13, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(most, device="cuda")
    first = torch.cumsum(had, 0) - had
    at = (first[:, None] + col[None]).clamp(max=total + granted)
    table = torch.where(col[None] < had[:, None], order[at], torch.full_like(order[at], -1))
    free = order[total:].contiguous()
    return {"case": case, "past": past, "new": new, "table": table.to(torch.int32).contiguous(), "free": free,
            "free_count": torch.tensor([free.numel()], dtype=torch.int32, device="cuda"),
            "tokens": B * case["new_most"]}  # room for every request's most


def _prepare_attn(case, seed):
    g = _gen(seed)
    B, n, H, KH, D, page = (case[x] for x in ("requests", "new", "heads", "kv_heads", "dim", "page"))
    lens = _lengths(case, seed) + n
    most = int(lens.max())
    per = (lens + page - 1) // page
    width = int(per.max())
    pages = int(per.sum()) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    per = per.cuda()
    first = torch.cumsum(per, 0) - per
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col[None]).clamp(max=pages - 1)
    table = torch.where(col[None] < per[:, None], order[at], torch.full_like(order[at], -1)).contiguous()
    gain, mid = _channels(g, KH, D)
    kq, ksz = _pool(pages, KH, page, D, case["group"])
    vq, vsz = _pool(pages, KH, page, D, case["group"])
    step = max(1, (1 << 26) // (KH * page * D))
    for a in range(0, pages, step):  # a stretch of pages at a time, to stay small
        m = min(step, pages - a)
        q, kz = _codes(_randn(g, m, KH, page, D) * gain[None, :, None] + mid[None, :, None], case["group"])
        kq[a:a + m], ksz[a:a + m] = _pack_keys(q), kz
        q, vz = _codes(_randn(g, m, KH, page, D), case["group"])
        vq[a:a + m], vsz[a:a + m] = _pack_values(q), vz
    return {"case": case, "q": _randn(g, B * n, H, D), "kq": kq, "ksz": ksz, "vq": vq, "vsz": vsz, "table": table,
            "lens": lens.to(torch.int32).cuda(),
            "starts": (torch.arange(B + 1, device="cuda") * n).to(torch.int32),
            "most": most, "scale": 1.0 / math.sqrt(D)}


def prepare(case, seed):
    return {"rope": _prepare_rope, "append": _prepare_append, "plan": _prepare_plan, "attn": _prepare_attn}[case["kind"]](case, seed)


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _rope_plain(s):
    c = s["case"]

    def one(x, gain):
        if gain is not None:
            x = x * (1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)) * gain
        angle = s["positions"].double()[:, None] * s["inv"].double()[None]
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        r = c["rot"]
        y = x[..., :r]
        if c["interleaved"]:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., r:]], -1)

    return one(s["q"], s["q_gain"]), one(s["k"], s["k_gain"])


def _append_plain(s):
    c = s["case"]
    page, at = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    q, sz = _codes(s["k"], c["group"])
    s["kq"][page, :, at], s["ksz"][page, :, at] = _pack_keys(q), sz
    q, sz = _codes(s["v"], c["group"])
    s["vq"][page, :, at], s["vsz"][page, :, at] = _pack_values(q), sz
    k = _values(_unpack_keys(s["kq"][page, :, at]), s["ksz"][page, :, at])
    v = _values(_unpack_values(s["vq"][page, :, at]), s["vsz"][page, :, at])
    return k, v


def _plan_plain(s):
    page = s["case"]["page"]
    past, new, table, T = s["past"].long(), s["new"].long(), s["table"], s["tokens"]
    B = past.numel()
    had = (past + page - 1) // page
    need = (past + new + page - 1) // page - had
    start = torch.cumsum(need, 0) - need
    top = s["free_count"].long()
    col = torch.arange(table.shape[1], device=table.device)[None]
    fresh = (col >= had[:, None]) & (col < (had + need)[:, None])
    take = (top - 1 - (start[:, None] + col - had[:, None])).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][take], table))
    starts = torch.zeros(B + 1, dtype=torch.long, device=table.device)
    starts[1:] = torch.cumsum(new, 0)
    t = torch.arange(T, device=table.device)
    b = (torch.searchsorted(starts, t, right=True) - 1).clamp(max=B - 1)
    live = t < starts[-1]
    pos = torch.where(live, past[b] + t - starts[b], torch.zeros_like(t))
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    slot = torch.where(live, slot, torch.full_like(slot, -1))
    i32 = torch.int32
    return {"table": table, "lens": (past + new).to(i32), "starts": starts.to(i32), "positions": pos.to(i32),
            "slots": slot.to(i32), "free": (top - need.sum()).to(i32)}


def _attn_plain(s):
    c = s["case"]
    B, n, H, KH, D, page = (c[x] for x in ("requests", "new", "heads", "kv_heads", "dim", "page"))
    L = s["most"]
    width = (L + page - 1) // page
    at = s["table"][:, :width].clamp(min=0).long()

    def rows(words, sz, unpack):  # [B, KH, width * page, D] of every request, padded to the longest
        x = _values(unpack(words[at]), sz[at])
        return x.transpose(1, 2).reshape(B, KH, width * page, D)

    k, v = rows(s["kq"], s["ksz"], _unpack_keys), rows(s["vq"], s["vsz"], _unpack_values)
    q = s["q"].reshape(B, n, KH, H // KH, D).permute(0, 2, 3, 1, 4).reshape(B, KH, H // KH * n, D)
    w = torch.matmul(q * s["scale"], k.transpose(-1, -2)).reshape(B, KH, H // KH, n, width * page)
    last = s["lens"].long()[:, None] - n + torch.arange(n, device=q.device)[None]
    t = torch.arange(width * page, device=q.device)
    seen = t <= last[..., None]
    if c["window"]:
        seen &= t > last[..., None] - c["window"]
    w = w.masked_fill(~seen[:, None, None], float("-inf"))
    w = torch.exp(w - w.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    v = v.masked_fill(~(t < s["lens"].long()[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(w.reshape(B, KH, H // KH * n, width * page), v)
    return o.reshape(B, KH, H // KH, n, D).permute(0, 3, 1, 2, 4).reshape(B * n, H, D)


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------

def _rope_own(gq4, s):
    return gq4.head_norm_rope(s["q"], s["k"], s["positions"], s["inv"], q_gain=s["q_gain"], k_gain=s["k_gain"],
                              eps=1e-6, interleaved=s["case"]["interleaved"])


def _append_own(gq4, s):
    cache = (s["kq"], s["ksz"], s["vq"], s["vsz"], s["case"]["group"])
    gq4.kv_append(s["k"], s["v"], s["slots"], *cache)
    return gq4.kv_gather(s["slots"], *cache)


def _plan_own(gq4, s):
    lens, starts, positions, slots, free = gq4.kv_plan(s["past"], s["new"], s["table"], s["free"], s["free_count"],
                                                       s["tokens"], s["case"]["page"])
    return {"table": s["table"], "lens": lens, "starts": starts, "positions": positions, "slots": slots, "free": free}


def _attn_own(gq4, s):
    return gq4.kv_attention(s["q"], s["starts"], s["lens"], s["table"], s["kq"], s["ksz"], s["vq"], s["vsz"],
                            s["case"]["group"], scale=s["scale"], max_query=s["case"]["new"], max_len=s["most"],
                            window=s["case"]["window"])


def run(state):
    kind = state["case"]["kind"]
    if own:
        from int4_group_quantized_quant_gb300 import gq4
        return {"rope": _rope_own, "append": _append_own, "plan": _plan_own, "attn": _attn_own}[kind](gq4, state)
    return {"rope": _rope_plain, "append": _append_plain, "plan": _plan_plain, "attn": _attn_plain}[kind](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    kind = case["kind"]
    if kind == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 8 * n + 4 * case["tokens"], "flops": 8 * n}
    if kind == "append":
        n = 2 * case["tokens"] * case["kv_heads"] * case["dim"]
        return {"bytes": 2 * (4 * n + n / 2 + 8 * n / case["group"]) + 8 * case["tokens"], "flops": 10 * n}
    if kind == "plan":
        B = case["requests"]
        T = B * case["new_most"]
        return {"bytes": 8 * B + 8 * B + 8 * T + 6 * T / case["page"], "flops": 0}
    H, KH, D, n = case["heads"], case["kv_heads"], case["dim"], case["new"]
    tokens = pairs = 0
    for past in _lengths(case, 0).tolist():
        first = max(0, past + 1 - case["window"]) if case["window"] else 0
        tokens += past + n - first
        w = case["window"] or past + n
        # query j sees min(past + 1 + j, w) keys
        full = min(n, max(0, past + n + 1 - w)) if case["window"] else 0
        pairs += full * w + (n - full) * (past + 1) + (n - full) * (n - full - 1) // 2
    rows = case["requests"] * n * H * D
    per = 2 * KH * (D / 2 + 8 * D / case["group"])
    return {"bytes": tokens * per + 8 * rows + 4 * tokens / case["page"], "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _rope_exact(s):
    c = s["case"]
    out = []
    for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
        x = x.double()
        if gain is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt() * gain.double()
        y = x.clone()
        for i in range(c["rot"] // 2):
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rot"] // 2)
            turn = torch.polar(torch.ones_like(s["positions"].double()), s["positions"].double() * s["inv"][i].double())
            z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
            y[..., a], y[..., b] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _attn_exact(s):
    c = s["case"]
    n, H, KH, D, page = (c[x] for x in ("new", "heads", "kv_heads", "dim", "page"))
    J = D // 32
    d = torch.arange(D, device="cuda")
    k_word, k_bit = (d % 32 // 8) * J + d // 32, 4 * (d % 8)
    v_half = (d % 32 // 4) * J + d // 32
    v_word, v_bit = v_half // 2, 16 * (v_half % 2) + 4 * (d % 4)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lens"].tolist()):
        pos = torch.arange(length, device="cuda")
        pg, at = s["table"][b, pos // page].long(), pos % page
        for h in range(KH):
            kv = []
            for words, sz, word, bit in ((s["kq"], s["ksz"], k_word, k_bit), (s["vq"], s["vsz"], v_word, v_bit)):
                code = (words[pg, h, at].long()[:, word] >> bit) % 16
                p = sz[pg, h, at].double()[:, d // c["group"]]
                kv.append((code.double() - p[..., 1]) * p[..., 0])
            for r in range(h * (H // KH), (h + 1) * (H // KH)):
                x = s["q"][b * n:(b + 1) * n, r].double() @ kv[0].T * s["scale"]
                gap = (length - n + torch.arange(n, device="cuda"))[:, None] - pos[None]
                x[gap < 0] = -math.inf
                if c["window"]:
                    x[gap >= c["window"]] = -math.inf
                out[b * n:(b + 1) * n, r] = torch.softmax(x, -1) @ kv[1]
    return out


def exact(case, seed):
    if case["kind"] in ("append", "plan"):
        return None  # codes and whole numbers: no such values
    return {"rope": _rope_exact, "attn": _attn_exact}[case["kind"]](prepare(case, seed))
