"""Plain 64-bit restatements of the operators between the QKV product and the
output projection, and the paged cache's layout in numpy, for the tests.

The cache's quantiser is restated in binary32 (its codes are decided there,
one rounding per step); everything else is float64.
"""

from __future__ import annotations

import math

import numpy as np

F32_TINY = np.float32(np.finfo(np.float32).tiny)


# ---------------------------------------------------------------------------
# Layout: codes [..., D] uint8 <-> rows of D/8 words
# ---------------------------------------------------------------------------

def places(D, keys):
    """(word, bit) of every code of a row."""
    d = np.arange(D)
    J = D // 32
    if keys:
        return (d % 32 // 8) * J + d // 32, 4 * (d % 8)
    h = (d % 32 // 4) * J + d // 32
    return h // 2, 16 * (h % 2) + 4 * (d % 4)


def pack(codes, keys):
    D = codes.shape[-1]
    word, bit = places(D, keys)
    out = np.zeros(codes.shape[:-1] + (D // 8,), np.uint32)
    for d in range(D):
        out[..., word[d]] |= codes[..., d].astype(np.uint32) << np.uint32(bit[d])
    return out


def unpack(words, keys):
    D = words.shape[-1] * 8
    word, bit = places(D, keys)
    return ((words[..., word] >> bit.astype(np.uint32)) & 15).astype(np.uint8)


def values(codes, sz):
    """(code - zero) * scale in float64; sz [..., G, 2]."""
    G = sz.shape[-2]
    v = codes.astype(np.float64).reshape(codes.shape[:-1] + (G, codes.shape[-1] // G))
    sz = sz.astype(np.float64)
    return ((v - sz[..., 1:]) * sz[..., :1]).reshape(codes.shape)


def quantise(x, gs):
    """(codes, sz) of f32 rows [..., D]: the header's rule, one binary32 rounding per step."""
    x = np.asarray(x, np.float32)
    v = x.reshape(x.shape[:-1] + (x.shape[-1] // gs, gs))
    with np.errstate(all="ignore"):
        lo = v.min(-1, keepdims=True) + np.float32(0)
        hi = v.max(-1, keepdims=True) + np.float32(0)
        d = hi - lo
        s = d / np.float32(15)
        s = np.where(s < F32_TINY, np.float32(1), s)
        q = np.rint((v - lo) * (np.float32(1) / s))
        z = -lo / s
        bad = ~np.isfinite(d)
        q = np.where(bad, 0, np.clip(q, 0, 15))
    nan = np.float32(np.nan)
    sz = np.concatenate([np.where(bad, nan, s), np.where(bad, nan, z)], -1)
    return q.astype(np.uint8).reshape(x.shape), sz.astype(np.float32)


class Cache:
    """A pool of random codes, scales and zeros, as numpy arrays."""

    def __init__(self, rng, pages, heads, page, D, gs):
        self.page, self.gs, self.D = page, gs, D
        shape = (pages, heads, page)
        self.codes = [rng.integers(0, 16, shape + (D,), dtype=np.uint8) for _ in range(2)]
        self.sz = [np.stack([rng.uniform(0.05, 0.3, shape + (D // gs,)),
                             rng.uniform(6, 9, shape + (D // gs,))], -1).astype(np.float32) for _ in range(2)]

    def arrays(self):
        """Kq, K_sz, Vq, V_sz."""
        return (pack(self.codes[0], True), self.sz[0], pack(self.codes[1], False), self.sz[1])

    def rows(self, side, head, slots):
        pg, at = slots // self.page, slots % self.page
        return values(self.codes[side][pg, head, at], self.sz[side][pg, head, at])


# ---------------------------------------------------------------------------
# Operators
# ---------------------------------------------------------------------------

def norm_rope(x, gain, eps, positions, inv_freq, interleaved):
    """(y, size) in float64, x [T, H, D]; size bounds |y_a| + |y_b| before the rotation."""
    x = x.astype(np.float64)
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * gain.astype(np.float64)
    y, size = x.copy(), np.abs(x)
    half = 0 if inv_freq is None else len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        # the product of a 31-bit and a 24-bit number, reduced without loss in long double
        turn = np.longdouble(1) * positions.astype(np.longdouble) * np.longdouble(inv_freq[i])
        turn = np.fmod(turn, 2 * np.longdouble(math.pi) + np.longdouble(2.4492935982947064e-16))
        c, s = np.cos(turn).astype(np.float64)[:, None], np.sin(turn).astype(np.float64)[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


def plan(past, new, table, free, free_count, T, page):
    """The header's rule, request by request."""
    B, room = len(past), table.shape[1] * page
    table = table.copy()
    avail = min(max(int(free_count), 0), len(free))
    starts, lens = [0], []
    pos, slots = np.zeros(T, np.int32), np.full(T, -1, np.int32)
    row = taken = granted = 0
    refused_any = False
    for b in range(B):
        p, n = max(int(past[b]), 0), max(int(new[b]), 0)
        refused = past[b] < 0 or new[b] < 0 or p + n > room or row + n > T
        need = 0
        had = (p + page - 1) // page
        if not refused:
            need = (p + n + page - 1) // page - had
            if need and taken + need > avail:
                refused = True
            taken += need
        if not refused:
            for j in range(need):
                table[b, had + j] = free[avail - 1 - (taken - need + j)]
            if need:
                granted = taken
        elif n > 0 or past[b] < 0 or new[b] < 0:
            refused_any = True
        if not refused:
            for j in range(n):
                pos[row + j] = p + j
                slots[row + j] = table[b, (p + j) // page] * page + (p + j) % page
        row += n
        starts.append(min(row, T))
        lens.append(p if refused else p + n)
    return (table, np.array(lens, np.int32), np.array(starts, np.int32), pos, slots,
            np.array([avail - granted], np.int32), refused_any)


def attention(q, starts, lens, table, cache, scale, window=0):
    """(out, tol) in float64; rows of no request are NaN in out.

    tol bounds the kernels' error.  A weight's exponent w = scale * q . k is a sum of D products of
    f32 (or two fp16 pieces: 2^-22) factors, with the zero taken off afterwards, so its error is at
    most A * (D/8 + 8) * 2^-23, A = scale * sum |q| s (code + |z|), where each of at most D/8 matrix
    steps cuts at most one unit of 2^-23 of the running sum and 8 more cover the splits, the zero and
    the final products; the base-2 exponential adds 2^-22 and the exponent's own rounding |w| 2^-23.
    An error e in the exponents moves the output by at most 2 e max|v|; the sum over the keys adds
    the same kind of error to v itself, on terms of size s (8 + |z - 8|): 16 units per key block on
    random signs, and the split's 2^-22.
    """
    T, H, D = q.shape
    out, tol = np.full((T, H, D), np.nan), np.zeros((T, H, D))
    KH = cache.codes[0].shape[1]
    R = H // KH
    for b in range(len(lens)):
        n, L = int(starts[b + 1] - starts[b]), int(lens[b])
        if n == 0:
            continue
        rows = slice(int(starts[b]), int(starts[b]) + n)
        last = L - n + np.arange(n)
        first = max(0, int(last[0]) + 1 - window) if window else 0
        t = np.arange(first, L)
        out[rows] = 0.0
        if not len(t):
            continue
        slots = table[b, t // cache.page].astype(np.int64) * cache.page + t % cache.page
        pg, at = slots // cache.page, slots % cache.page
        seen = t[None] <= last[:, None]
        if window:
            seen &= t[None] > last[:, None] - window
        some = seen.any(-1)
        seen = np.repeat(seen[some], R, 0)                                   # [rows * R, keys]
        for kh in range(KH):
            k, v = cache.rows(0, kh, slots), cache.rows(1, kh, slots)
            sz = np.repeat(cache.sz[0][pg, kh, at].astype(np.float64), cache.gs, axis=-2)
            size = np.abs(sz[..., 0]) * (cache.codes[0][pg, kh, at] + np.abs(sz[..., 1]))
            vz = np.repeat(cache.sz[1][pg, kh, at].astype(np.float64), cache.gs, axis=-2)
            vsize = (np.abs(vz[..., 0]) * (8 + np.abs(vz[..., 1] - 8))).max(-1)
            x = q[rows, kh * R:(kh + 1) * R].astype(np.float64)[some].reshape(-1, D)
            w = scale * (x @ k.T)
            A = np.where(seen, abs(scale) * (np.abs(x) @ size.T), 0).max(-1)
            wmax = np.where(seen, np.abs(w), 0).max(-1)
            vmax = np.where(seen, vsize[None], 0).max(-1)
            w = np.where(seen, w, -np.inf)
            w = np.exp(w - w.max(-1, keepdims=True))
            o = (w @ v) / w.sum(-1, keepdims=True)
            e = A * (D / 8 + 8) * 2.0 ** -23 + 2.0 ** -22 + wmax * 2.0 ** -23
            bound = 2 * e * vmax + 16 * 2.0 ** -23 * vmax
            at_rows = np.arange(rows.start, rows.stop)[some]
            out[at_rows, kh * R:(kh + 1) * R] = o.reshape(-1, R, D)
            tol[at_rows, kh * R:(kh + 1) * R] = bound.reshape(-1, R, 1)
    return out, tol
