"""Drafted trees and long streams over the paged 4-bit cache, measured.

Kinds of cases:
  append - a step's queries rotated, its keys rotated and quantised into the cache, its values quantised, one pass;
  tree   - positions and ancestor bits of drafted trees from their parents;
  attn   - attention over the cache of drafted trees, or behind a sliding window with first tokens that stay visible;
  accept - the accepted path of every tree moved to the end of its request, the pages left over given back.

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
        # one decode step of 61 requests, normalised heads
        _case("append_step", "append", tokens=61, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False, norm=True,
              group=128, page=16),
        # a long prompt, heads as the projection leaves them
        _case("append_prompt", "append", tokens=16381, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False,
              norm=False, group=64, page=64),
        # the tree of one request: latency of the smallest call
        _case("tree_one", "tree", requests=1, nodes=15, past_most=4096, words=1, window=0, sinks=0),
        # a full server's trees, with a window
        _case("tree_many", "tree", requests=256, nodes=60, past_most=4096, words=2, window=2048, sinks=4),
        # one request's tree behind a short context: latency
        _case("attn_tree_one", "attn", requests=1, new=15, tree=True, past_least=776, past_most=776, heads=32,
              kv_heads=8, dim=128, group=128, page=16, window=0, sinks=0),
        # the ordinary verification step: a ragged batch
        _case("attn_tree_batch", "attn", requests=32, new=26, tree=True, past_least=500, past_most=4096, heads=32,
              kv_heads=8, dim=128, group=128, page=16, window=0, sinks=0),
        # wide trees behind long documents, finer groups
        _case("attn_tree_wide", "attn", requests=4, new=64, tree=True, past_least=8000, past_most=16000, heads=32,
              kv_heads=8, dim=128, group=64, page=64, window=0, sinks=0),
        # one endless stream: latency
        _case("attn_sink_one", "attn", requests=1, new=1, tree=False, past_least=5000, past_most=5000, heads=32,
              kv_heads=8, dim=128, group=128, page=16, window=1024, sinks=4),
        # a decode step of many streams, short and long
        _case("attn_sink_batch", "attn", requests=64, new=1, tree=False, past_least=200, past_most=60000, heads=32,
              kv_heads=8, dim=128, group=128, page=16, window=4096, sinks=4),
        # chunks of prompts after earlier chunks, the finest groups
        _case("attn_sink_chunk", "attn", requests=3, new=1021, tree=False, past_least=1000, past_most=16000, heads=32,
              kv_heads=8, dim=128, group=32, page=16, window=2048, sinks=64),
        # after the verification of a few requests' trees
        _case("accept_step", "accept", requests=16, nodes=15, past_most=2048, kv_heads=8, dim=128, group=128, page=16),
        # the same on a full server
        _case("accept_many", "accept", requests=256, nodes=60, past_most=2048, kv_heads=8, dim=128, group=64, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    kind = rng.choice(["append", "append", "tree", "attn", "attn", "attn", "attn", "accept"])
    dim = rng.choice([64, 96, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 5, 8])
    ratio = rng.choice([1, 2, 4, 5, 7, 8])
    group = rng.choice([g for g in (32, 64, 96, 128, 256) if dim % g == 0])
    page = rng.choice([16, 32, 64, 128])
    if kind == "append":
        most = 16381 * 48 * 128 // ((ratio + 2) * kv * dim)
        return {"kind": kind, "tokens": _log(rng, 1, min(most, 40000)), "heads": ratio * kv, "kv_heads": kv, "dim": dim,
                "rot": rng.choice([dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.4,
                "norm": rng.random() < 0.5, "group": group, "page": page}
    if kind == "tree":
        nodes = _log(rng, 1, 200)
        return {"kind": kind, "requests": _log(rng, 1, 256 * 60 // nodes), "nodes": nodes, "past_most": _log(rng, 1, 8192),
                "words": (nodes + 31) // 32 + rng.choice([0, 1]), "window": rng.choice([0, 0, 1, 3, 1000]),
                "sinks": rng.choice([0, 4, 100])}
    if kind == "accept":
        nodes = _log(rng, 1, 200)
        most = max(1, 256 * 60 * 8 * 128 // (nodes * kv * dim))
        return {"kind": kind, "requests": _log(rng, 1, min(256, most)), "nodes": nodes, "past_most": _log(rng, 1, 2048),
                "kv_heads": kv, "dim": dim, "group": group, "page": page}
    heads = ratio * kv
    tree = rng.random() < 0.5
    new = _log(rng, 1, 200) if tree else 1 if rng.random() < 0.5 else _log(rng, 1, 1500)
    window = rng.choice([0, 0, _log(rng, 1, 4096)]) if tree else _log(rng, 1, 4096)
    sinks = rng.choice([0, 4]) if tree else _log(rng, 1, 100)
    past = _log(rng, 1, 60000)
    # within the listed chunks' products and rows, and the listed caches' bytes
    flops, rows, codes = 4 * 128 * 32 * 3 * 1021 * 2000, 3 * 1021 * 32 * 128, 64 * 4096 * 8 * 128
    new = max(1, min(new, rows // (heads * dim)))
    seen = min(past, window) if window else past
    cap = max(1, min(flops // (4 * heads * dim * new) - new, codes // (kv * dim) - new))
    if seen > cap:
        past = seen = cap
    most = max(1, min(flops // (4 * heads * dim * new * (seen + new)), rows // (heads * dim * new),
                      codes // (kv * dim * (seen + new + sinks))))
    return {"kind": kind, "requests": _log(rng, 1, min(64, most)), "new": new, "tree": tree,
            "past_least": rng.choice([0, past // 2]), "past_most": past, "heads": heads, "kv_heads": kv, "dim": dim,
            "group": group, "page": page, "window": window, "sinks": sinks}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0x6752 + int(seed))
    return g


def _host_gen(seed):
    """For lengths and trees, which work() needs too."""
    g = torch.Generator()
    g.manual_seed(0x52 + int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


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


def _pool(pages, kv_heads, page, dim, group):
    words = torch.zeros(pages, kv_heads, page, dim // 8, dtype=torch.int32, device="cuda")
    sz = torch.zeros(pages, kv_heads, page, dim // group, 2, device="cuda")
    return words, sz


def _filled(g, pages, kv_heads, page, dim, group):
    """Pools of keys and values, every page written."""
    gain, mid = _channels(g, kv_heads, dim)
    kq, ksz = _pool(pages, kv_heads, page, dim, group)
    vq, vsz = _pool(pages, kv_heads, page, dim, group)
    step = max(1, (1 << 26) // (kv_heads * page * dim))
    for a in range(0, pages, step):  # a stretch of pages at a time, to stay small
        m = min(step, pages - a)
        q, kz = _codes(_randn(g, m, kv_heads, page, dim) * gain[None, :, None] + mid[None, :, None], group)
        kq[a:a + m], ksz[a:a + m] = _pack_keys(q), kz
        q, vz = _codes(_randn(g, m, kv_heads, page, dim), group)
        vq[a:a + m], vsz[a:a + m] = _pack_values(q), vz
    return {"kq": kq, "ksz": ksz, "vq": vq, "vsz": vsz}


def _prepare_append(case, seed):
    g = _gen(seed)
    T, H, KH, D, page = (case[x] for x in ("tokens", "heads", "kv_heads", "dim", "page"))
    qkv = _randn(g, T, H + 2 * KH, D)  # q, k and v side by side, as one projection leaves them
    gain, mid = _channels(g, KH, D)
    qkv[:, H:H + KH] *= gain
    qkv[:, H:H + KH] += mid
    half = case["rot"] // 2
    inv = (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
    start = int(torch.randint(0, 200001, (1,), generator=_host_gen(seed)))
    pages = (T + page - 1) // page + 7
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    t = torch.arange(T, device="cuda")
    kq, ksz = _pool(pages, KH, page, D, case["group"])
    vq, vsz = _pool(pages, KH, page, D, case["group"])
    return {"case": case, "q": qkv[:, :H], "k": qkv[:, H:H + KH], "v": qkv[:, H + KH:], "inv": inv,
            "positions": (start + t).to(torch.int32), "slots": (order[t // page] * page + t % page).to(torch.int32),
            "q_gain": 1.0 + 0.2 * _randn(g, D) if case["norm"] else None,
            "k_gain": 1.0 + 0.2 * _randn(g, D) if case["norm"] else None,
            "kq": kq, "ksz": ksz, "vq": vq, "vsz": vsz}


def _parents(sizes, g):
    """Drafted trees, one after the other: a node's parent is one of the eight before it; -1: the last token of the past."""
    i = torch.cat([torch.arange(n) for n in sizes])
    u = torch.rand(i.numel(), generator=g)
    return (i - 1 - (u * i.clamp(max=8)).long()).to(torch.int32)


def _starts(sizes):
    return torch.cat([torch.zeros(1, dtype=torch.long), torch.as_tensor(sizes).cumsum(0)]).to(torch.int32)


def _prepare_tree(case, seed):
    g = _host_gen(seed)
    B = case["requests"]
    sizes = torch.randint((case["nodes"] + 1) // 2, case["nodes"] + 1, (B,), generator=g)
    past = torch.randint(0, case["past_most"] + 1, (B,), generator=g)
    T = B * case["nodes"]  # room for every request's most; rows of no node stay as they are
    parents = torch.zeros(T, dtype=torch.int32)
    parents[:int(sizes.sum())] = _parents(sizes.tolist(), g)
    return {"case": case, "parents": parents.cuda(), "starts": _starts(sizes).cuda(),
            "lens": (past + sizes).to(torch.int32).cuda(),
            "positions": torch.zeros(T, dtype=torch.int32, device="cuda"),
            "tree": torch.zeros(T, case["words"], dtype=torch.int32, device="cuda")}


def _lengths(case, seed):
    """The requests' past lengths of an attention case and, of a tree, its parents, on the host."""
    g = _host_gen(seed)
    past = torch.randint(case["past_least"], case["past_most"] + 1, (case["requests"],), generator=g)
    return past, _parents([case["new"]] * case["requests"], g) if case["tree"] else None


def _prepare_attn(case, seed):
    g = _gen(seed)
    B, n, H, KH, D, page = (case[x] for x in ("requests", "new", "heads", "kv_heads", "dim", "page"))
    past, parents = _lengths(case, seed)
    lens = past + n
    # pages that no query sees are gone
    first = (past + 1 - case["window"]).clamp(min=0) // page if case["window"] else torch.zeros_like(past)
    kept = (case["sinks"] + page - 1) // page if case["window"] else 0
    col = torch.arange(int((lens.max() + page - 1) // page))[None]
    live = (col < ((lens + page - 1) // page)[:, None]) & ((col >= first[:, None]) | (col < kept))
    pages = int(live.sum()) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = (live.flatten().cumsum(0) - 1).reshape(live.shape).clamp(min=0).cuda()
    table = torch.where(live.cuda(), order[at], torch.full_like(order[at], -1)).contiguous()
    s = {"case": case, "q": _randn(g, B * n, H, D), "table": table, "lens": lens.to(torch.int32).cuda(),
         "starts": (torch.arange(B + 1, device="cuda") * n).to(torch.int32), "most": int(lens.max()),
         "scale": 1.0 / math.sqrt(D), "tree": None, "positions": None, **_filled(g, pages, KH, page, D, case["group"])}
    if case["tree"]:  # what the step has from its trees' parents
        s["positions"], s["tree"] = _tree_bits(parents.cuda(), s["starts"], s["lens"], (n + 31) // 32, case["window"],
                                               case["sinks"])
    return s


def _paths(case, seed):
    """Past lengths and the accepted paths: from node 0 on, each step 1 to 8 nodes on, some of them or none accepted."""
    g = _host_gen(seed)
    B, n = case["requests"], case["nodes"]
    past = torch.randint(0, case["past_most"] + 1, (B,), generator=g)
    step = torch.randint(1, 9, (B, min(n, 16)), generator=g)
    step[:, 0] = 1
    path = step.cumsum(1) - 1
    count = torch.minimum((path < n).sum(1), torch.randint(0, path.shape[1] + 1, (B,), generator=g))
    return past, path.clamp(max=n - 1), count


def _prepare_accept(case, seed):
    g = _gen(seed)
    B, n, page = case["requests"], case["nodes"], case["page"]
    past, path, count = _paths(case, seed)
    lens = past + n
    col = torch.arange(int((lens.max() + page - 1) // page))[None]
    live = col < ((lens + page - 1) // page)[:, None]
    pages = int(live.sum()) + 13
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = (live.flatten().cumsum(0) - 1).reshape(live.shape).clamp(min=0).cuda()
    table = torch.where(live.cuda(), order[at], torch.full_like(order[at], -1)).contiguous()
    free = torch.full((B * ((case["past_most"] + n + page - 1) // page) + 13,), -1, dtype=torch.int32, device="cuda")
    free[:13] = order[pages - 13:]
    return {"case": case, "path": path.to(torch.int32).cuda(), "count": count.to(torch.int32).cuda(),
            "starts": (torch.arange(B + 1, device="cuda") * n).to(torch.int32), "lens": lens.to(torch.int32).cuda(),
            "table": table, "free": free, "free_count": torch.tensor([13], dtype=torch.int32, device="cuda"),
            "slots": _path_slots(past.cuda(), path.shape[1], count.cuda(), table, page),
            "k": torch.zeros(path.numel(), case["kv_heads"], case["dim"], device="cuda"),
            "v": torch.zeros(path.numel(), case["kv_heads"], case["dim"], device="cuda"),
            **_filled(g, pages, case["kv_heads"], page, case["dim"], case["group"])}


def _path_slots(past, most, count, table, page):
    """Where the accepted rows come to lie, to read them back; -1 behind the last."""
    i = torch.arange(most, device="cuda")[None]
    t = past[:, None] + i
    at = (t // page).clamp(max=table.shape[1] - 1)
    slot = table.gather(1, at).long() * page + t % page
    return torch.where(i < count[:, None], slot, torch.full_like(slot, -1)).flatten().to(torch.int32)


def prepare(case, seed):
    return {"append": _prepare_append, "tree": _prepare_tree, "attn": _prepare_attn,
            "accept": _prepare_accept}[case["kind"]](case, seed)


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _append_plain(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv"].double()[None]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def turned(x, gain):  # in 64 bits, rounded once: a key next to a border of two codes falls on its own side
        x = x.double()
        if gain is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain.double()
        r = c["rot"]
        y = x[..., :r]
        if c["interleaved"]:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., r:]], -1).float()

    page, at = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    q, sz = _codes(turned(s["k"], s["k_gain"]), c["group"])
    s["kq"][page, :, at], s["ksz"][page, :, at] = _pack_keys(q), sz
    q, sz = _codes(s["v"], c["group"])
    s["vq"][page, :, at], s["vsz"][page, :, at] = _pack_values(q), sz
    return turned(s["q"], s["q_gain"]), *_read(s)


def _read(s):
    """The rows at s["slots"], as the values that their codes stand for."""
    slots = s["slots"].long().clamp(min=0)
    page, at = slots // s["case"]["page"], slots % s["case"]["page"]
    return (_values(_unpack_keys(s["kq"][page, :, at]), s["ksz"][page, :, at]),
            _values(_unpack_values(s["vq"][page, :, at]), s["vsz"][page, :, at]))


def _tree_bits(parents, starts, lens, words, window, sinks):
    """(positions [T], bits [T, words]): bit i of a node's row is node i of its request, an ancestor or itself, that the
    window leaves it."""
    T, N = parents.numel(), 32 * words
    t = torch.arange(T, device=parents.device)
    b = (torch.searchsorted(starts, t, right=True) - 1).clamp(max=lens.numel() - 1)
    i = (t - starts[b]).clamp(max=N - 1)
    # up[b, i, j]: j is i or an ancestor of it; the parents' matrix with itself, squared until every path is in it
    up = torch.eye(N, device=parents.device).repeat(lens.numel(), 1, 1)
    has = (parents >= 0) & (t < starts[-1])
    up[b[has], i[has].long(), parents[has].long()] = 1.0
    for _ in range(8):
        up = (torch.matmul(up, up) > 0).float()
    depth = up.sum(-1).long() - 1
    past = lens.long() - (starts[1:] - starts[:-1])
    if window:
        near = (depth[:, :, None] - depth[:, None, :] < window) | ((past[:, None] + depth)[:, None, :] < sinks)
        up = up * near
    bits = (up[b, i.long()].long().reshape(T, words, 32) << torch.arange(32, device=parents.device)).sum(-1)
    bits = torch.where(bits >= 2**31, bits - 2**32, bits)
    return (past[b] + depth[b, i.long()]).to(torch.int32), bits.to(torch.int32)


def _tree_plain(s):
    c = s["case"]
    positions, bits = _tree_bits(s["parents"], s["starts"], s["lens"], c["words"], c["window"], c["sinks"])
    live = torch.arange(positions.numel(), device=positions.device) < s["starts"][-1]
    return torch.where(live, positions, s["positions"]), torch.where(live[:, None], bits, s["tree"])


def _attn_plain(s):
    c = s["case"]
    B, n, H, KH, D, page = (c[x] for x in ("requests", "new", "heads", "kv_heads", "dim", "page"))
    w, dev = c["window"], s["q"].device
    lens = s["lens"].long()
    past = lens - n
    # the positions that some query sees, padded to the longest: the window's, and the first tokens before it
    lo = (past + 1 - w).clamp(min=0) if w else torch.zeros_like(past)
    S = c["sinks"] if w else 0
    t = lo[:, None] + torch.arange(min(s["most"], w + n) if w else s["most"], device=dev)
    there = t < lens[:, None]
    first = torch.arange(S, device=dev).expand(B, S)
    t, there = torch.cat([first, t], 1), torch.cat([first < lo[:, None], there], 1)
    pg = s["table"].gather(1, (t // page).clamp(max=s["table"].shape[1] - 1)).long().clamp(min=0)
    at = t % page

    def rows(words, sz, unpack):  # [B, KH, keys, D]
        return _values(unpack(words[pg, :, at]), sz[pg, :, at]).transpose(1, 2)

    k, v = rows(s["kq"], s["ksz"], _unpack_keys), rows(s["vq"], s["vsz"], _unpack_values)
    q = s["q"].reshape(B, n, KH, H // KH, D).permute(0, 2, 3, 1, 4).reshape(B, KH, H // KH * n, D)
    x = torch.matmul(q * s["scale"], k.transpose(-1, -2)).reshape(B, KH, H // KH, n, -1)
    if c["tree"]:
        p, new = s["positions"].long().reshape(B, n, 1), (t - past[:, None])[:, None]
        word = s["tree"].reshape(B, n, -1).gather(2, (new // 32).clamp(0, s["tree"].shape[1] - 1).expand(B, n, -1))
        bit = ((word >> (new % 32)) & 1).bool()
        old = (t[:, None] > p - w) | (t[:, None] < S) if w else torch.ones_like(bit)
        seen = torch.where(new < 0, old, bit)
    else:
        p = (past[:, None] + torch.arange(n, device=dev))[..., None]
        seen = t[:, None] <= p
        if w:
            seen &= (t[:, None] > p - w) | (t[:, None] < S)
    seen &= there[:, None]
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x = x / x.sum(-1, keepdim=True)
    v = v.masked_fill(~there[:, None, :, None], 0.0)
    o = torch.matmul(x.reshape(B, KH, H // KH * n, -1), v)
    return o.reshape(B, KH, H // KH, n, D).permute(0, 3, 1, 2, 4).reshape(B * n, H, D)


def _accept_plain(s):
    c = s["case"]
    page, table = c["page"], s["table"]
    lens, count = s["lens"].long(), s["count"].long()
    past = lens - (s["starts"][1:] - s["starts"][:-1])
    i = torch.arange(s["path"].shape[1], device=table.device)[None]
    taken = i < count[:, None]
    src, dst = past[:, None] + s["path"], past[:, None] + i
    b = torch.arange(lens.numel(), device=table.device)[:, None].expand_as(taken)[taken]
    src, dst = src[taken], dst[taken]
    ps, pd = table[b, src // page].long(), table[b, dst // page].long()
    for pool in ("kq", "ksz", "vq", "vsz"):
        s[pool][pd, :, dst % page] = s[pool][ps, :, src % page]  # every row is read before any is written
    left = past + count
    col = torch.arange(table.shape[1], device=table.device)[None]
    over = (col >= ((left + page - 1) // page)[:, None]) & (col < ((lens + page - 1) // page)[:, None])
    back = table[over]
    top = s["free_count"].long()
    s["free"][top + torch.arange(back.numel(), device=table.device)] = back
    return {"lens": left.to(torch.int32), "free": s["free"], "free_count": (top + back.numel()).to(torch.int32),
            "rows": [torch.where((s["slots"] >= 0)[:, None, None], x, y) for x, y in zip(_read(s), (s["k"], s["v"]))]}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------

def _cache(s):
    return s["kq"], s["ksz"], s["vq"], s["vsz"], s["case"]["group"]


def _append_own(gq4, s):
    q = gq4.kv_rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv"], s["slots"], *_cache(s), q_gain=s["q_gain"],
                           k_gain=s["k_gain"], eps=1e-6, interleaved=s["case"]["interleaved"])
    return q, *gq4.kv_gather(s["slots"], *_cache(s))


def _tree_own(gq4, s):
    c = s["case"]
    return gq4.kv_tree(s["parents"], s["starts"], s["lens"], c["words"], window=c["window"], sinks=c["sinks"],
                       positions=s["positions"], tree=s["tree"])


def _attn_own(gq4, s):
    c = s["case"]
    return gq4.kv_attention(s["q"], s["starts"], s["lens"], s["table"], *_cache(s), scale=s["scale"], max_query=c["new"],
                            max_len=s["most"], window=c["window"], sinks=c["sinks"], tree=s["tree"],
                            positions=s["positions"])


def _accept_own(gq4, s):
    lens, count = gq4.kv_accept(s["path"], s["count"], s["starts"], s["lens"], s["table"], s["free"], s["free_count"],
                                *_cache(s))
    return {"lens": lens, "free": s["free"], "free_count": count, "rows": gq4.kv_gather(s["slots"], *_cache(s), s["k"], s["v"])}


def run(state):
    kind = state["case"]["kind"]
    if own:
        from int4_group_quantized_quant_gb300 import gq4
        return {"append": _append_own, "tree": _tree_own, "attn": _attn_own, "accept": _accept_own}[kind](gq4, state)
    return {"append": _append_plain, "tree": _tree_plain, "attn": _attn_plain, "accept": _accept_plain}[kind](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    kind = case["kind"]
    if kind == "tree":
        T = case["requests"] * (case["nodes"] + (case["nodes"] + 1) // 2) / 2
        return {"bytes": T * (4 + 4 + 4 * case["words"]) + 8 * case["requests"], "flops": 0}
    D = case["dim"]
    row = 2 * case["kv_heads"] * (D / 2 + 8 * D / case["group"])  # a token's codes, scales and zeros
    if kind == "append":
        q, kv = case["tokens"] * case["heads"] * D, 2 * case["tokens"] * case["kv_heads"] * D
        # written to the cache and read back
        return {"bytes": 8 * q + 2 * (4 * kv + case["tokens"] * row) + 12 * case["tokens"], "flops": 8 * q + 14 * kv}
    if kind == "accept":
        taken = int(_paths(case, 0)[2].sum())
        # moved, and read back
        return {"bytes": taken * (3 * row + 8 * case["kv_heads"] * D) + 16 * case["requests"], "flops": 0}
    H, n, w = case["heads"], case["new"], case["window"]
    pasts, parents = _lengths(case, 0)
    up = 0  # pairs of a node and an ancestor or itself
    if case["tree"]:
        depth = []
        for t, p in enumerate(parents.tolist()):
            depth.append(1 if p < 0 else depth[t - t % n + p] + 1)
        up = sum(depth)
    tokens = pairs = 0
    for past in pasts.tolist():
        first = max(0, past + 1 - w) if w else 0
        kept = min(case["sinks"], first) if w else 0
        tokens += past + n - first + kept
        if case["tree"]:
            pairs += n * (past - first + kept)
        else:  # query j sees min(past + 1 + j, w) keys and the first ones
            full = min(n, max(0, past + n + 1 - w)) if w else 0
            pairs += full * w + (n - full) * (past + 1) + (n - full) * (n - full - 1) // 2 + n * kept
    rows = case["requests"] * n * H * D
    return {"bytes": tokens * row + 8 * rows + 4 * tokens / case["page"], "flops": 4 * D * H * (pairs + up)}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _append_exact(s):
    c = s["case"]
    x = s["q"].double()
    if s["q_gain"] is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt() * s["q_gain"].double()
    y = x.clone()
    for i in range(c["rot"] // 2):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rot"] // 2)
        turn = torch.polar(torch.ones_like(s["positions"].double()), s["positions"].double() * s["inv"][i].double())
        z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
        y[..., a], y[..., b] = z.real, z.imag
    return y, None, None  # codes: no such values


def _attn_exact(case, seed):
    s = _prepare_attn(case, seed)
    n, H, KH, D, page = (case[x] for x in ("new", "heads", "kv_heads", "dim", "page"))
    J = D // 32
    d = torch.arange(D, device="cuda")
    k_word, k_bit = (d % 32 // 8) * J + d // 32, 4 * (d % 8)
    v_half = (d % 32 // 4) * J + d // 32
    v_word, v_bit = v_half // 2, 16 * (v_half % 2) + 4 * (d % 4)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    pasts, parents = _lengths(case, seed)
    for b, past in enumerate(pasts.tolist()):
        # rows of keys that each query sees, from the parents themselves
        first = max(0, past + 1 - case["window"]) if case["window"] else 0
        kept = min(case["sinks"], first) if case["window"] else 0
        pos = torch.cat([torch.arange(kept), torch.arange(first, past + n)])
        seen = torch.zeros(n, pos.numel(), dtype=torch.bool)
        depth = []
        for j in range(n):
            if case["tree"]:
                up = int(parents[b * n + j])
                depth.append(past if up < 0 else depth[up] + 1)
                seen[j] = pos < past
                node = j
                while node >= 0:
                    if not case["window"] or depth[j] - depth[node] < case["window"] or depth[node] < case["sinks"]:
                        seen[j, kept + past - first + node] = True
                    node = int(parents[b * n + node])
            else:
                depth.append(past + j)
                seen[j] = pos <= past + j
            if case["window"]:
                gone = (pos <= depth[j] - case["window"]) & (pos >= case["sinks"])
                seen[j] &= ~(gone & (pos < past)) if case["tree"] else ~gone
        pos, seen = pos.cuda(), seen.cuda()
        pg, at = s["table"][b, pos // page].long(), pos % page
        for h in range(KH):
            kv = []
            for words, sz, word, bit in ((s["kq"], s["ksz"], k_word, k_bit), (s["vq"], s["vsz"], v_word, v_bit)):
                code = (words[pg, h, at].long()[:, word] >> bit) % 16
                p = sz[pg, h, at].double()[:, d // case["group"]]
                kv.append((code.double() - p[..., 1]) * p[..., 0])
            for r in range(h * (H // KH), (h + 1) * (H // KH)):
                x = s["q"][b * n:(b + 1) * n, r].double() @ kv[0].T * s["scale"]
                out[b * n:(b + 1) * n, r] = torch.softmax(x.masked_fill(~seen, -math.inf), -1) @ kv[1]
    return out


def exact(case, seed):
    if case["kind"] == "append":
        return _append_exact(_prepare_append(case, seed))
    return _attn_exact(case, seed) if case["kind"] == "attn" else None  # the others: whole numbers and copies
