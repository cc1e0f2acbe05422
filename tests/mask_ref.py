"""Plain 64-bit restatements of the attention with first tokens that stay visible and with drafted trees, of the trees'
book-keeping and of accepting a path, for the tests."""

from __future__ import annotations

import numpy as np

from tests import kv_ref as R


def tree(parents, starts, lens, words, window=0, sinks=0):
    """(positions, bits uint32 [T, words], refused) node by node; rows of no request are 0."""
    T = len(parents)
    pos, bits = np.zeros(T, np.int32), np.zeros((T, words), np.uint32)
    refused = False
    for b in range(len(lens)):
        lo, n = int(starts[b]), int(starts[b + 1] - starts[b])
        past = int(lens[b]) - n
        own = parents[lo:lo + n]
        if n > 32 * words or past < 0 or any(not -1 <= p < i for i, p in enumerate(own)):
            refused = True
            continue
        depth = []
        for i, p in enumerate(own):
            depth.append(0 if p < 0 else depth[p] + 1)
            pos[lo + i] = past + depth[i]
            j = i
            while j >= 0:
                if not window or depth[i] - depth[j] < window or past + depth[j] < sinks:
                    bits[lo + i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
                j = own[j]
    return pos, bits, refused


def sight(n, L, window, sinks, bits=None, positions=None):
    """Which of a request's L keys its n queries see, [n, L]."""
    past, t = L - n, np.arange(max(L, 0))
    if bits is None:
        p = past + np.arange(n)[:, None]
        old = t[None] <= p
    else:
        p = past + np.zeros((n, 1), int)
        if window:
            p = np.clip(positions[:, None], past, L - 1)
        old = np.broadcast_to(t[None] < past, (n, len(t)))
    seen = old & ((t[None] > p - window) | (t[None] < sinks)) if window else old.copy()
    if bits is not None:
        for i in range(min(n, 32 * bits.shape[1])):
            if past + i >= 0:
                seen[:, past + i] = (bits[:, i // 32] >> np.uint32(i % 32)) & 1
    return seen


def attention(q, starts, lens, table, cache, scale, window=0, sinks=0, bits=None, positions=None):
    """(out, tol) in float64; rows of no request are NaN in out.  tol as kv_ref.attention derives it: the same sums, over
    the keys that a row sees."""
    T, H, D = q.shape
    out, tol = np.full((T, H, D), np.nan), np.zeros((T, H, D))
    KH = cache.codes[0].shape[1]
    G = H // KH
    for b in range(len(lens)):
        lo, n, L = int(starts[b]), int(starts[b + 1] - starts[b]), int(lens[b])
        if n == 0:
            continue
        out[lo:lo + n] = 0.0
        seen = sight(n, L, window, sinks, None if bits is None else bits[lo:lo + n],
                     None if positions is None else positions[lo:lo + n])
        t = np.nonzero(seen.any(0))[0]
        if not len(t):
            continue
        slots = table[b, t // cache.page].astype(np.int64) * cache.page + t % cache.page
        some = seen.any(1)
        rows = np.arange(lo, lo + n)[some]
        seen = np.repeat(seen[some][:, t], G, 0)
        pg, at = slots // cache.page, slots % cache.page
        for kh in range(KH):
            k, v = cache.rows(0, kh, slots), cache.rows(1, kh, slots)
            sz = np.repeat(cache.sz[0][pg, kh, at].astype(np.float64), cache.gs, axis=-2)
            size = np.abs(sz[..., 0]) * (cache.codes[0][pg, kh, at] + np.abs(sz[..., 1]))
            vz = np.repeat(cache.sz[1][pg, kh, at].astype(np.float64), cache.gs, axis=-2)
            vsize = (np.abs(vz[..., 0]) * (8 + np.abs(vz[..., 1] - 8))).max(-1)
            x = q[rows][:, kh * G:(kh + 1) * G].astype(np.float64).reshape(-1, D)
            w = scale * (x @ k.T)
            A = np.where(seen, abs(scale) * (np.abs(x) @ size.T), 0).max(-1)
            wmax = np.where(seen, np.abs(w), 0).max(-1)
            vmax = np.where(seen, vsize[None], 0).max(-1)
            w = np.where(seen, w, -np.inf)
            w = np.exp(w - w.max(-1, keepdims=True))
            o = np.where(seen, w, 0) @ np.where(seen.any(0)[:, None], v, 0) / w.sum(-1, keepdims=True)
            e = A * (D / 8 + 8) * 2.0 ** -23 + 2.0 ** -22 + wmax * 2.0 ** -23
            bound = 2 * e * vmax + 16 * 2.0 ** -23 * vmax
            out[rows, kh * G:(kh + 1) * G] = o.reshape(-1, G, D)
            tol[rows, kh * G:(kh + 1) * G] = bound.reshape(-1, G, 1)
    return out, tol


def accept(path, count, starts, lens, table, free, free_count, n_pages, page):
    """(lens, free, free_count, moves [(request, from, to)], refused): the header's rule, request by request."""
    free, lens_out, moves, back = free.copy(), [], [], []
    refused = False
    for b in range(len(lens)):
        n, L, c = int(starts[b + 1] - starts[b]), int(lens[b]), int(count[b])
        past = L - n
        nodes = [int(path[b][i]) for i in range(c)] if path is not None and 0 <= c <= path.shape[1] else list(range(max(c, 0)))
        span = range(past // page, (L + page - 1) // page)
        bad = n < 0 or past < 0 or L > table.shape[1] * page or not 0 <= c <= n or (path is not None and c > path.shape[1])
        bad = bad or any(not (nodes[i - 1] if i else -1) < x < n for i, x in enumerate(nodes))
        bad = bad or (n > 0 and any(not 0 <= table[b, i] < n_pages for i in span))
        if bad:
            refused = True
            lens_out.append(L)
            continue
        moves += [(b, past + x, past + i) for i, x in enumerate(nodes) if x != i]
        lens_out.append(past + c)
        back += [int(table[b, i]) for i in range((past + c + page - 1) // page, (L + page - 1) // page)]
    top = min(max(int(free_count), 0), len(free))
    fit = back[:len(free) - top]
    free[top:top + len(fit)] = fit
    return np.array(lens_out, np.int32), free, top + len(fit), moves, refused or len(fit) < len(back)


def random_parents(g, n, reach=8):
    """A tree whose nodes come after their parents; a few roots."""
    return np.array([int(g.integers(max(-1, i - reach), i)) if i else -1 for i in range(n)], np.int32)
