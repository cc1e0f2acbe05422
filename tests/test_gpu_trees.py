"""GPU tests of rotation and append in one pass, of drafted trees' book-keeping and of accepting a path, against the
64-bit restatements of tests/kv_ref.py and tests/mask_ref.py, and of a whole speculative loop."""

import numpy as np
import pytest
import torch

from int4_group_quantized_quant_gb300 import inputs as I
from tests import kv_ref as R
from tests import mask_ref as M
from tests.gpu_util import dev, gq4_module, host, requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def gq4():
    g = gq4_module()
    g.device_error(clear=True)
    return g


def inv_freq(rot):
    return (10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)


def codes_of(arrays, slots, page):
    """([key codes, value codes], [key sz, value sz]) of slots, from host arrays of the four pools."""
    kq, ksz, vq, vsz = arrays
    pg, at = slots // page, slots % page
    return ([R.unpack(kq.view(np.uint32)[pg, :, at], True), R.unpack(vq.view(np.uint32)[pg, :, at], False)],
            [ksz[pg, :, at], vsz[pg, :, at]])


def check_rows(gq4, q, k, v, pos, inv, slots, cache, gs, page, qg, kg, inter, qr):
    """What one call has left, against 64 bits.

    A code is that of the key in 64 bits rounded to f32, exactly.  A value that codes stand for, lo + c s: the lower end
    is off by at most 9 roundings of |a| + |b| <= 2 A, A the largest of the row, the range by twice that, and the
    restatement's own four steps and the kernel's round by at most 5 units of the value each: 18 + 36 + 10 units of
    2^-24 A."""
    if q is not None:
        y, size = R.norm_rope(q, qg, 1e-6, pos, inv, inter)
        assert np.all(np.abs(qr - y) <= 16 * 2.0 ** -24 * size)
    y, size = R.norm_rope(k, kg, 1e-6, pos, inv, inter)
    live = slots >= 0
    codes, sz = codes_of([host(t) for t in cache], slots[live], page)
    want, want_sz = R.quantise(y.astype(np.float32)[live], gs)
    assert np.array_equal(codes[0], want)
    err = np.abs(R.values(codes[0], sz[0]) - R.values(want, want_sz))
    assert np.all(err <= 64 * 2.0 ** -24 * size[live].max(-1, keepdims=True))
    want, want_sz = R.quantise(v[live], gs)
    assert np.array_equal(codes[1], want) and np.array_equal(sz[1].view(np.uint32), want_sz.view(np.uint32))


APPENDS = [
    # T, H, KH, D, gs, page, rot, interleaved, q gain, k gain
    (1, 32, 8, 128, 128, 16, 128, False, True, True), (61, 32, 8, 128, 64, 16, 128, False, False, False),
    (33, 5, 5, 64, 32, 32, 64, True, True, True), (17, 7, 1, 64, 64, 64, 16, False, False, True),
    (40, 6, 3, 96, 96, 16, 96, False, True, True), (21, 3, 1, 96, 32, 128, 24, True, False, False),
    (9, 4, 2, 256, 64, 16, 256, False, True, True), (12, 2, 2, 256, 256, 256, 128, True, True, False),
    (25, 0, 4, 128, 32, 16, 128, False, False, True), (30, 16, 3, 256, 32, 16, 8, False, True, True),
    (700, 4, 5, 128, 128, 16, 128, False, True, True), (650, 9, 3, 64, 32, 16, 32, True, False, False),
    (50, 2, 2, 128, 32, 16, 0, False, True, True), (31, 1, 7, 96, 32, 16, 88, False, False, False),
    (401, 3, 2, 64, 64, 16, 64, False, True, True), (307, 0, 1, 256, 128, 32, 128, True, False, False),
    (305, 33, 17, 96, 96, 16, 48, False, False, True), (3, 200, 65, 64, 32, 16, 64, False, True, True),
    (4999, 2, 8, 128, 64, 16, 128, True, False, True),
]


@pytest.mark.parametrize("T,H,KH,D,gs,page,rot,inter,qn,kn", APPENDS)
def test_rope_append(gq4, T, H, KH, D, gs, page, rot, inter, qn, kn):
    g = I.rng(2500, T, H, KH, D, gs, rot)
    wide = g.standard_normal((T, H + 2 * KH + 1, D)).astype(np.float32)
    wide[:, H:H + KH] = wide[:, H:H + KH] * np.exp(0.3 * g.standard_normal((KH, D))) + 0.3 * g.standard_normal((KH, D))
    x = dev(wide)
    q, k, v = (wide[:, :H] if H else None), wide[:, H:H + KH], wide[:, H + KH:H + 2 * KH]
    pages = (T + page - 1) // page + 2
    slots = g.permutation(pages * page)[:T].astype(np.int32)
    pos = g.integers(0, 200000, T).astype(np.int32)
    qg, kg = (g.uniform(0.5, 1.5, D).astype(np.float32) if n else None for n in (qn and H, kn))
    inv = inv_freq(rot) if rot else None
    cache = gq4.kv_cache(pages, KH, page, D, gs)
    qr = gq4.kv_rope_append(x[:, :H] if H else None, x[:, H:H + KH], x[:, H + KH:H + 2 * KH], dev(pos) if rot else None,
                            dev(inv) if rot else None, dev(slots), *cache, gs, q_gain=None if qg is None else dev(qg),
                            k_gain=None if kg is None else dev(kg), interleaved=inter)
    torch.cuda.synchronize()
    assert gq4.device_error() == 0
    assert np.array_equal(host(x), wide)
    check_rows(gq4, q, k, v, pos, inv, slots, cache, gs, page, qg, kg, inter, host(qr) if H else None)


BORDER = [(128, 128, 128, False, False), (128, 32, 128, False, True), (64, 64, 32, True, False), (96, 96, 96, False, False),
          (256, 64, 128, True, True)]


@pytest.mark.parametrize("D,gs,rot,inter,norm", BORDER)
def test_keys_next_to_a_border(gq4, D, gs, rot, inter, norm):
    """Keys whose rotated values lie on the borders of two codes but for the roundings of their inputs: each code is
    that of the value in 64 bits."""
    keys_next_to_a_border(gq4, D, gs, rot, inter, norm, 0, 2)


@pytest.mark.parametrize("power", [-100, -51, -49, 49, 51, 100])
@pytest.mark.parametrize("D,gs,rot,inter,norm", [c for c in BORDER if not c[4]])
def test_keys_next_to_a_border_of_any_size(gq4, D, gs, rot, inter, norm, power):
    keys_next_to_a_border(gq4, D, gs, rot, inter, norm, power, 5)


def keys_next_to_a_border(gq4, D, gs, rot, inter, norm, power, KH):
    T, page = 200, 16
    g = I.rng(2501, D, gs, rot)
    inv = inv_freq(rot)
    pos = g.integers(0, 50000, T).astype(np.int32)
    gain = np.exp2(g.integers(-1, 2, D)).astype(np.float32) if norm else None
    # the rotated row: a group's ends, and halves between two codes; turned back
    y = g.integers(0, 15, (T, KH, D // gs, gs)) + 0.5
    y[..., 0], y[..., -1] = 0, 15
    y = (y - 7).reshape(T, KH, D) / 8
    half, x = rot // 2, y.copy()
    ang = pos[:, None].astype(np.float64) * inv.astype(np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, half), slice(half, rot))
    x[..., a], x[..., b] = y[..., a] * c + y[..., b] * s, y[..., b] * c - y[..., a] * s
    k = (x / (gain if norm else 1.0) * 2.0 ** power).astype(np.float32)
    v = g.standard_normal((T, KH, D)).astype(np.float32)
    slots = g.permutation(T + 8)[:T].astype(np.int32)
    cache = gq4.kv_cache((T + 8) // page, KH, page, D, gs)
    gq4.kv_rope_append(None, dev(k), dev(v), dev(pos), dev(inv), dev(slots), *cache, gs, interleaved=inter,
                       k_gain=dev(gain) if norm else None)
    torch.cuda.synchronize()
    check_rows(gq4, None, k, v, pos, inv, slots, cache, gs, page, None, gain, inter, None)


def test_rope_append_like_the_two_calls(gq4):
    """Queries in place in a fused row; the other columns and skipped slots stay; V bit for bit as kv_append's."""
    T, H, KH, D, gs, page = 37, 8, 2, 128, 64, 16
    g = I.rng(2502)
    wide = g.standard_normal((T, H + 2 * KH, D)).astype(np.float32)
    slots = g.permutation(80)[:T].astype(np.int32)
    slots[::5] = -1
    pos, inv = g.integers(0, 9000, T).astype(np.int32), inv_freq(D)
    gain = g.uniform(0.5, 1.5, D).astype(np.float32)
    x, z = dev(wide), dev(wide)
    one, two = gq4.kv_cache(5, KH, page, D, gs), gq4.kv_cache(5, KH, page, D, gs)
    out = gq4.kv_rope_append(x[:, :H], x[:, H:H + KH], x[:, H + KH:], dev(pos), dev(inv), dev(slots), *one, gs,
                             q_gain=dev(gain), k_gain=dev(gain), q_out=x[:, :H])
    assert out.data_ptr() == x.data_ptr()
    qr, kr = gq4.head_norm_rope(z[:, :H], z[:, H:H + KH], dev(pos), dev(inv), q_gain=dev(gain), k_gain=dev(gain))
    gq4.kv_append(kr, z[:, H + KH:], dev(slots), *two, gs)
    torch.cuda.synchronize()
    assert torch.equal(x[:, H:], z[:, H:])
    y, size = R.norm_rope(wide[:, :H], gain, 1e-6, pos, inv, False)
    assert np.all(np.abs(host(x[:, :H]).astype(np.float64) - host(qr)) <= 32 * 2.0 ** -24 * size)
    assert torch.equal(one[2], two[2]) and torch.equal(one[3].view(torch.int32), two[3].view(torch.int32))
    check_rows(gq4, None, wide[:, H:H + KH], wide[:, H + KH:], pos, inv, slots, one, gs, page, None, gain, False, None)
    used = np.zeros(80, bool)
    used[slots[slots >= 0]] = True
    assert np.all(host(one[1]).transpose(0, 2, 1, 3, 4).reshape(80, -1)[~used] == 0)
    assert gq4.device_error() == 0


def test_far_positions_and_huge_frequencies(gq4):
    """Positions up to 2^31 - 1: queries and values hold; frequencies beyond all sense stay bounded, NaN ones are NaN."""
    T, D = 5, 64
    g = I.rng(2504)
    pos = np.array([2**31 - 1, 2**30 + 12345, 2**20 + 1, 7, 0], np.int32)
    q, k, v = (g.standard_normal((T, 2, D)).astype(np.float32) for _ in range(3))
    cache = gq4.kv_cache(1, 2, 16, D, 32)
    slots = np.arange(T, dtype=np.int32)
    qr = gq4.kv_rope_append(dev(q), dev(k), dev(v), dev(pos), dev(inv_freq(D)), dev(slots), *cache, 32)
    y, size = R.norm_rope(q, None, 0, pos, inv_freq(D), False)
    # an angle is a 64-bit product, off by 2^-53 of it: 2^-22 at 2^31
    assert np.all(np.abs(host(qr) - y) <= (16 * 2.0 ** -24 + pos[:, None, None] * 2.0 ** -53) * size)
    kr = host(gq4.kv_gather(dev(slots), *cache, 32)[0])
    y, size = R.norm_rope(k, None, 0, pos, inv_freq(D), False)
    step = host(cache[1])[0, :, :T, :, 0].transpose(1, 0, 2).repeat(32, -1)
    assert np.all(np.abs(kr - y) <= 0.5 * step + 64 * 2.0 ** -22 * size)
    inv = inv_freq(D)
    inv[3], inv[5] = 1e30, np.nan
    qr = host(gq4.kv_rope_append(dev(q), dev(k), dev(v), dev(pos), dev(inv), dev(slots), *cache, 32))
    bad = np.zeros(D, bool)
    bad[[5, 5 + D // 2]] = True
    assert np.isnan(qr[..., bad]).all() and np.all(np.abs(qr[..., ~bad]) <= 2 * np.abs(q).max())
    assert gq4.device_error(clear=True) == 1 << 3


def test_rope_append_marks_what_is_wrong(gq4):
    """A slot outside the pool, groups that are not finite: bits 6 and 3, nothing else touched; zero rows; no tokens."""
    T, KH, D, gs, page = 6, 2, 64, 32, 16
    g = I.rng(2503)
    k, v = (g.standard_normal((T, KH, D)).astype(np.float32) for _ in range(2))
    pos, inv = np.arange(T, dtype=np.int32), inv_freq(D)
    slots = np.array([3, 64, 5, 7, 2**31 - 1, 9], np.int32)
    k[2, 1, 3], v[3, 0, 40] = np.inf, np.nan
    k[5] = 0
    cache = gq4.kv_cache(4, KH, page, D, gs)
    q = g.standard_normal((T, 3, D)).astype(np.float32)
    qr = gq4.kv_rope_append(dev(q), dev(k), dev(v), dev(pos), dev(inv), dev(slots), *cache, gs)
    torch.cuda.synchronize()
    assert gq4.device_error(clear=True) == (1 << 6 | 1 << 3)
    y, size = R.norm_rope(q, None, 0, pos, inv, False)
    assert np.all(np.abs(host(qr) - y) <= 16 * 2.0 ** -24 * size)
    sz = host(cache[1])[0].transpose(1, 0, 2, 3), host(cache[3])[0].transpose(1, 0, 2, 3)   # [slot, head, group, 2]
    assert np.isnan(sz[0][5, 1]).all()      # the pair (3, 35): both groups
    assert np.isfinite(sz[0][5, 0]).all() and np.isfinite(sz[1][5]).all()
    assert np.isnan(sz[1][7, 0, 1]).all() and np.isfinite(sz[1][7, 0, 0]).all() and np.isfinite(sz[0][7]).all()
    assert np.array_equal(sz[0][9], np.broadcast_to(np.array([1, 0], np.float32), (KH, 2, 2)))
    assert np.all(sz[0][[0, 1, 2, 4, 6, 8]] == 0)
    gq4.kv_rope_append(dev(q[:0]), dev(k[:0]), dev(v[:0]), dev(pos[:0]), dev(inv), dev(slots[:0]), *cache, gs)
    assert gq4.device_error() == 0


# ---------------------------------------------------------------------------

@pytest.mark.parametrize("sizes,words", [([1], 1), ([15], 1), ([32, 1, 33, 64, 0, 7], 2), ([256, 0, 255, 1], 8), ([5] * 700, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (2, 9), (0, 4)])
def test_trees(gq4, sizes, words, window, sinks):
    g = I.rng(2510, len(sizes), words, window)
    starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    T = int(starts[-1]) + 3
    parents = np.concatenate([M.random_parents(g, n, 1 if b % 3 == 2 else 8) for b, n in enumerate(sizes)] + [np.full(3, 7)])
    lens = (np.array(sizes) + g.integers(0, 20, len(sizes))).astype(np.int32)
    pos, tree = torch.full((T,), -9, dtype=torch.int32, device="cuda"), torch.full((T, words), -9, dtype=torch.int32, device="cuda")
    gq4.kv_tree(dev(parents.astype(np.int32)), dev(starts), dev(lens), words, window=window, sinks=sinks, positions=pos, tree=tree)
    want_pos, want, refused = M.tree(parents, starts, lens, words, window, sinks)
    assert not refused and gq4.device_error() == 0
    live = T - 3
    assert np.array_equal(host(pos)[:live], want_pos[:live]) and np.array_equal(host(tree).view(np.uint32)[:live], want[:live])
    assert np.all(host(pos)[live:] == -9) and np.all(host(tree)[live:] == -9)


def test_trees_that_are_none(gq4):
    """A parent that comes later, is the node itself, is below -1; too many nodes; more nodes than tokens; rows out of T."""
    sizes = [4, 4, 4, 33, 4, 3]
    starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    T = int(starts[-1])
    parents = np.concatenate([M.random_parents(I.rng(1), n) for n in sizes])
    parents[1], parents[6], parents[8] = 2, 2, -2
    lens = np.array([9, 9, 9, 40, 3, 9], np.int32)
    pos, tree = gq4.kv_tree(dev(parents), dev(starts), dev(lens), 1)
    want_pos, want, refused = M.tree(parents, starts, lens, 1)
    assert refused and gq4.device_error(clear=True) == 1 << 10
    assert np.array_equal(host(pos), want_pos) and np.array_equal(host(tree).view(np.uint32), want)
    starts[-1] = T + 5
    pos, tree = gq4.kv_tree(dev(parents), dev(starts), dev(lens), 2)
    assert gq4.device_error(clear=True) == 1 << 10
    assert np.all(host(pos)[starts[5]:] == 0) and np.all(host(tree)[starts[5]:] == 0)
    starts[-1], starts[0] = T, -4
    pos, tree = gq4.kv_tree(dev(parents), dev(starts), dev(lens), 2)
    assert gq4.device_error(clear=True) == 1 << 10
    assert np.all(host(pos)[:4] == 0)


class Accept:
    """Requests with drafted rows in a pool of random rows, and paths through them."""

    def __init__(self, sizes, KH=3, D=64, gs=32, page=16, past=60, spare=2, seed=0):
        g = I.rng(2520, len(sizes), KH, D, gs, page, seed)
        B = len(sizes)
        self.page, self.gs, self.KH, self.D = page, gs, KH, D
        self.starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        self.lens = (g.integers(0, past, B) + sizes).astype(np.int32)
        per = (self.lens + page - 1) // page
        self.pages = int(per.sum()) + spare
        order = g.permutation(self.pages).astype(np.int32)
        self.table = np.full((B, int(per.max()) + 1), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :per[b]] = order[at:at + per[b]]
            at += per[b]
        self.free = np.full(self.pages, -7, np.int32)
        self.free[:spare] = order[at:]
        self.count_free = spare
        most = max(max(sizes), 1)
        self.path = np.full((B, most), 10**6, np.int32)
        self.counts = np.zeros(B, np.int32)
        for b, n in enumerate(sizes):
            self.counts[b] = int(g.integers(0, n + 1)) if b % 4 else n if b % 8 else 0
            self.path[b, :self.counts[b]] = np.sort(g.permutation(n)[:self.counts[b]])
        self.cache = R.Cache(g, self.pages, KH, page, D, gs)

    def want(self, path="own"):
        lens, free, count, moves, refused = M.accept(self.path if path == "own" else path, self.counts, self.starts, self.lens,
                                                     self.table, self.free, self.count_free, self.pages, self.page)
        arrays = [a.copy() for a in self.cache.arrays()]
        old = [a.copy() for a in arrays]
        for b, src, dst in moves:
            (ps, s), (pd, d) = ((self.table[b, t // self.page], t % self.page) for t in (src, dst))
            for a, o in zip(arrays, old):
                a[pd, :, d] = o[ps, :, s]
        return lens, free, count, arrays, refused

    def check(self, gq4, path="own", **kw):
        lens, free, count, arrays, refused = self.want(path)
        cache, free_dev = [dev(a) for a in self.cache.arrays()], dev(self.free)
        p = self.path if path == "own" else path
        got = gq4.kv_accept(None if p is None else dev(p), dev(self.counts), dev(self.starts), dev(self.lens), dev(self.table),
                            free_dev, dev(np.array([self.count_free], np.int32)), *cache, self.gs, **kw)
        torch.cuda.synchronize()
        assert gq4.device_error(clear=True) == (1 << 11 if refused else 0)
        assert np.array_equal(host(got[0]), lens) and host(got[1]).tolist() == [count]
        assert np.array_equal(host(free_dev), free)
        for a, c in zip(arrays, cache):
            assert np.array_equal(host(c).view(np.uint32), a.view(np.uint32))


@pytest.mark.parametrize("sizes,kw", [
    ([15], {}), ([1, 0, 60, 17, 16, 5, 31, 2, 33], dict(KH=8, D=128, gs=128)), ([40, 3, 0, 9], dict(KH=5, D=96, gs=32, page=32)),
    ([7, 100, 64], dict(KH=1, D=256, gs=64, page=64)), ([300, 4, 280], dict(KH=2, D=64, gs=64, page=128)),
    ([int(n) for n in np.arange(1500) % 9], dict(KH=1)), ([20] * 40, dict(KH=9, D=96, gs=96)),
])
def test_accept(gq4, sizes, kw):
    Accept(sizes, **kw).check(gq4)
    a = Accept(sizes, seed=1, **kw)
    a.check(gq4, path=None)
    a.check(gq4, workspace=torch.full((gq4.lib.gq4_kv_accept_workspace_bytes(len(sizes)),), 77, dtype=torch.uint8, device="cuda"))


def test_accept_refuses(gq4):
    """Counts and paths that cannot be, pages outside the pool, lengths past the table: those requests stay as they are."""
    a = Accept([10] * 14, past=40)
    a.counts[:] = 4
    a.path[:, :4] = [0, 3, 5, 9]
    a.counts[1], a.counts[2] = -1, 11
    a.path[3, 2], a.path[4, 1], a.path[5, 3], a.path[6, 0] = 3, 0, 10, -1
    past = a.lens - 10
    a.table[7, past[7] // 16] = -1
    a.table[8, (a.lens[8] - 1) // 16] = a.pages
    a.lens[9] = 9
    a.lens[10] = a.table.shape[1] * 16 + 1
    a.lens[11] = -3
    a.check(gq4)
    # no room on the list for all that comes back; a count above it
    b = Accept([100, 90, 80], past=5)
    b.counts[:] = 0
    b.free, b.count_free = b.free[:6], 2
    b.check(gq4)
    b.count_free = 9
    b.check(gq4)
    b.free, b.count_free = b.free[:0], 0
    b.check(gq4)


def test_accept_in_place_and_in_a_graph(gq4):
    """Lengths and count advanced in place; a captured call replayed on new state gives what an eager one does."""
    a = Accept([33, 7, 0, 60, 12], KH=8, D=128, gs=64)
    lens, free, count, arrays, _ = a.want()
    args = [dev(a.path), dev(a.counts), dev(a.starts), dev(a.lens), dev(a.table), dev(a.free),
            dev(np.array([a.count_free], np.int32)), *[dev(x) for x in a.cache.arrays()], a.gs]
    keep = [t.clone() if isinstance(t, torch.Tensor) else t for t in args]

    def call():
        return gq4.kv_accept(*args, seq_lens_out=args[3], free_count_out=args[6])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call()
    for run in (call, graph.replay, graph.replay):
        for t, k in zip(args, keep):
            if isinstance(t, torch.Tensor):
                t.copy_(k)
        run()
        torch.cuda.synchronize()
        assert np.array_equal(host(args[3]), lens) and host(args[6]).tolist() == [count]
        assert np.array_equal(host(args[5]), free)
        for x, c in zip(arrays, args[7:11]):
            assert np.array_equal(host(c).view(np.uint32), x.view(np.uint32))
    assert gq4.device_error() == 0


def test_calls_on_another_stream(gq4):
    """The outputs and workspaces that calls allocate for another stream, while that stream is still busy."""
    a = Accept([33, 7, 60], KH=2)
    lens, free, count, _, _ = a.want()
    args = [dev(a.path), dev(a.counts), dev(a.starts), dev(a.lens), dev(a.table), dev(a.free),
            dev(np.array([a.count_free], np.int32)), *[dev(x) for x in a.cache.arrays()], a.gs]
    parents = np.concatenate([M.random_parents(I.rng(3), n) for n in (33, 7, 60)])
    up = dev(parents)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    pos, tree = gq4.kv_tree(up, args[2], args[3], 2, stream=side)
    got = gq4.kv_accept(*args, stream=side)
    filler = [torch.full((200,), 123, dtype=torch.int32, device="cuda") for _ in range(50)]
    torch.cuda.synchronize()
    assert len(filler) == 50
    want_pos, want, _ = M.tree(parents, a.starts, a.lens, 2)
    assert np.array_equal(host(pos), want_pos) and np.array_equal(host(tree).view(np.uint32), want)
    assert np.array_equal(host(got[0]), lens) and host(got[1]).tolist() == [count]


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 4)])
@pytest.mark.parametrize("graph", [False, True])
def test_speculative_loop(gq4, window, sinks, graph):
    """A prompt and six steps of drafted trees: plan, tree, rotation and append, attention, accept; captured or not.
    What the cache holds in the end is what a plain decode of the accepted tokens would have written, every attention is
    that of the rows in the cache, and no page is lost."""
    H, KH, D, gs, page, B, n, words, pages, width = 8, 2, 64, 32, 16, 3, 11, 1, 40, 12
    g = I.rng(2530, window)
    inv = inv_freq(D)
    gain = g.uniform(0.5, 1.5, D).astype(np.float32)
    cache = gq4.kv_cache(pages, KH, page, D, gs)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count = dev(np.arange(pages, dtype=np.int32)), dev(np.array([pages], np.int32))
    lens = dev(np.zeros(B, np.int32))
    dinv, dgain = dev(inv), dev(gain)
    tokens = [[] for _ in range(B)]             # (position, k, v) of what stays

    # the prompt: a line of tokens
    news = [20, 5, 33]
    T = sum(news)
    x = g.standard_normal((T, H + 2 * KH, D)).astype(np.float32)
    _, starts, pos, slots, _ = gq4.kv_plan(lens, dev(np.array(news, np.int32)), table, free, count, T, page, seq_lens=lens,
                                           free_count_out=count)
    d = dev(x)
    gq4.kv_rope_append(d[:, :H], d[:, H:H + KH], d[:, H + KH:], pos, dinv, slots, *cache, gs, k_gain=dgain)
    row = 0
    for b, m in enumerate(news):
        tokens[b] += [(i, x[row + i, H:H + KH], x[row + i, H + KH:]) for i in range(m)]
        row += m

    T = B * n
    new = dev(np.full(B, n, np.int32))
    xin, parents = torch.zeros((T, H + 2 * KH, D), device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    path, counts = torch.zeros((B, n), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = {}
    ws = torch.empty(gq4.kv_attention_workspace_bytes(T, H, KH, D, tree=True), dtype=torch.uint8, device="cuda")

    def draft():
        _, st, _, slt, _ = gq4.kv_plan(lens, new, table, free, count, T, page, seq_lens=lens, free_count_out=count)
        p, tree = gq4.kv_tree(parents, st, lens, words, window=window, sinks=sinks)
        qr = gq4.kv_rope_append(xin[:, :H], xin[:, H:H + KH], xin[:, H + KH:], p, dinv, slt, *cache, gs, k_gain=dgain)
        out = gq4.kv_attention(qr, st, lens, table, *cache, gs, scale=D ** -0.5, max_query=n, window=window, sinks=sinks,
                               tree=tree, positions=p, workspace=ws)
        kept.update(starts=st, positions=p, slots=slt, q=qr, out=out, tree=tree)

    def accept():
        gq4.kv_accept(path, counts, kept["starts"], lens, table, free, count, *cache, gs, seq_lens_out=lens, free_count_out=count)

    graphs = None
    if graph:
        side, graphs = torch.cuda.Stream(), [torch.cuda.CUDAGraph() for _ in range(2)]
        torch.cuda.synchronize()
        for gr, f in zip(graphs, (draft, accept)):
            with torch.cuda.stream(side):
                with torch.cuda.graph(gr, stream=side):
                    f()
    for step in range(6):
        x = g.standard_normal((T, H + 2 * KH, D)).astype(np.float32)
        up = np.concatenate([M.random_parents(g, n, 4) for _ in range(B)])
        xin.copy_(dev(x))
        parents.copy_(dev(up))
        graphs[0].replay() if graph else draft()
        torch.cuda.synchronize()
        assert gq4.device_error() == 0
        now, st, pos = host(lens), host(kept["starts"]), host(kept["positions"])
        assert now.tolist() == [len(t) + n for t in tokens]
        # the attention, on the rows that the cache holds
        tb = host(table)
        ks, vs = gq4.kv_gather(dev(np.concatenate([tb[b, t // page] * page + t % page for b in range(B)
                                                   for t in [np.arange(now[b])]]).astype(np.int32)), *cache, gs)
        ks, vs, qh, out = (host(t).astype(np.float64) for t in (ks, vs, kept["q"], kept["out"]))
        at = 0
        want_pos, bits, _ = M.tree(up, st, now, words, window, sinks)
        assert np.array_equal(pos, want_pos)
        for b in range(B):
            L, rows = int(now[b]), slice(int(st[b]), int(st[b + 1]))
            seen = M.sight(n, L, window, sinks, bits[rows], pos[rows])
            for h in range(H):
                w = D ** -0.5 * qh[rows, h] @ ks[at:at + L, h // (H // KH)].T
                w = np.where(seen, np.exp(w - np.where(seen, w, -np.inf).max(-1, keepdims=True)), 0)
                ref = w @ vs[at:at + L, h // (H // KH)] / w.sum(-1, keepdims=True)
                assert np.allclose(out[rows, h], ref, rtol=1e-4, atol=1e-4)
            at += L
        # a path from a root, from parent to child
        chosen = np.zeros((B, n), np.int32)
        taken = np.zeros(B, np.int32)
        for b in range(B):
            own, nodes = up[b * n:(b + 1) * n], []
            for _ in range(int(g.integers(0, 5))):
                below = [i for i in range(n) if own[i] == (nodes[-1] if nodes else -1)]
                if not below:
                    break
                nodes.append(int(g.choice(below)))
            chosen[b, :len(nodes)], taken[b] = nodes, len(nodes)
            tokens[b] += [(int(pos[b * n + i]), x[b * n + i, H:H + KH], x[b * n + i, H + KH:]) for i in nodes]
        path.copy_(dev(chosen))
        counts.copy_(dev(taken))
        graphs[1].replay() if graph else accept()
        torch.cuda.synchronize()
        assert gq4.device_error() == 0
        now, tb = host(lens), host(table)
        assert now.tolist() == [len(t) for t in tokens]
        held = [tb[b, :(now[b] + page - 1) // page].tolist() for b in range(B)]
        left = host(free)[:int(host(count)[0])].tolist()
        assert sorted(sum(held, []) + left) == list(range(pages))
    for b in range(B):
        t = np.arange(now[b])
        assert [p for p, _, _ in tokens[b]] == t.tolist()
        slots = tb[b, t // page] * page + t % page
        check_rows(gq4, None, np.stack([k for _, k, _ in tokens[b]]), np.stack([v for _, _, v in tokens[b]]),
                   t.astype(np.int32), inv, slots, cache, gs, page, None, gain, False, None)
