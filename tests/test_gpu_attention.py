"""GPU tests of the attention over the paged 4-bit cache (gq4_kv_attention)
against a float64 restatement (tests/kv_ref.py, which also derives the bound),
and of a decode loop of the operators together."""

import numpy as np
import pytest
import torch

import oracle
from int4_group_quantized_quant_gb300 import inputs as I
from tests import kv_ref as R
from tests.gpu_util import check_close, dev, gq4_module, host, requires_cuda, tol_fp32, wdev

pytestmark = [pytest.mark.gpu, requires_cuda]

FILL = -1234.5


@pytest.fixture(scope="module")
def gq4():
    g = gq4_module()
    g.device_error(clear=True)
    return g


class Setup:
    """Requests over a pool with scattered pages; unused slots and table entries hold rubbish."""

    def __init__(self, news, lens, H, KH, D, gs, page, window=0, pad=3, seed=0):
        g = I.rng(2200, sum(news), sum(lens), H, KH, D, gs, page, window, seed)
        per = [(n + page - 1) // page for n in lens]
        pages = sum(per) + 3
        self.cache = R.Cache(g, pages, KH, page, D, gs)
        order = g.permutation(pages)
        self.table = np.full((len(lens), max(max(per), 1) + 1), -5, np.int32)
        used = np.zeros((pages, page), bool)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
            for t in range(lens[b]):
                used[self.table[b, t // page], t % page] = True
        for side in range(2):  # slots that hold no key
            self.cache.sz[side][np.broadcast_to(~used[:, None], self.cache.sz[side].shape[:3])] = np.nan
        if window:  # pages wholly before the first visible key may be gone
            for b, n in enumerate(lens):
                for i in range(max(0, n - news[b] + 1 - window) // page):
                    self.table[b, i] = 10**9
        self.starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.T = int(self.starts[-1]) + pad
        self.q = g.standard_normal((self.T, H, D)).astype(np.float32)
        self.lens = np.asarray(lens, np.int32)
        self.news, self.window, self.gs, self.scale = news, window, gs, 1.0 / np.sqrt(D)

    def dev(self):
        return [dev(self.starts), dev(self.lens), dev(self.table), *[dev(a) for a in self.cache.arrays()], self.gs]

    def run(self, gq4, q=None, args=None, **kw):
        out = torch.full(self.q.shape, FILL, device="cuda")
        opts = dict(scale=self.scale, max_query=max(self.news), max_len=int(self.lens.max()), window=self.window,
                    out=out)
        opts.update(kw)
        gq4.kv_attention(dev(self.q) if q is None else q, *(args or self.dev()), **opts)
        torch.cuda.synchronize()
        return host(opts["out"])

    def check(self, got):
        ref, tol = R.attention(self.q, self.starts, self.lens, self.table, self.cache, self.scale, self.window)
        live = int(self.starts[-1])
        assert np.all(got[live:] == FILL), "rows of no request changed"
        if live == 0:
            return
        got, ref, tol = got[:live].astype(np.float64), ref[:live], tol[:live]
        assert np.all(np.isfinite(got))
        err = np.abs(got - ref)
        assert np.all(err <= tol), f"worst err/tol {float((err / np.maximum(tol, 1e-300)).max()):.3g}"
        assert np.linalg.norm(err) <= 1e-5 * np.linalg.norm(ref), np.linalg.norm(err) / np.linalg.norm(ref)


SHAPES = [
    # H, KH, D, gs, page
    (32, 8, 128, 128, 16), (4, 4, 64, 32, 16), (8, 1, 128, 32, 64), (6, 2, 96, 96, 32), (10, 2, 96, 32, 16),
    (7, 1, 256, 64, 128), (5, 1, 64, 64, 256), (3, 3, 256, 256, 16), (32, 2, 128, 64, 16), (40, 2, 64, 32, 64),
]


@pytest.mark.parametrize("H,KH,D,gs,page", SHAPES)
def test_single_tokens(gq4, H, KH, D, gs, page):
    """A decode step whose lengths end inside and at the edges of tiles and pages."""
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 255, 256, 257, 300]
    s = Setup([1] * len(lens), lens, H, KH, D, gs, page)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("H,KH,D,gs,page", SHAPES)
def test_ragged_queries(gq4, H, KH, D, gs, page):
    """Prompts, chunks, single tokens and idle requests side by side."""
    news, lens = [0, 3, 1, 17, 40, 0, 2, 65], [9, 3, 70, 17, 300, 0, 130, 66]
    s = Setup(news, lens, H, KH, D, gs, page)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("window", [1, 16, 50, 200])
@pytest.mark.parametrize("H,KH,D,gs,page", SHAPES[:4])
def test_window(gq4, H, KH, D, gs, page, window):
    news, lens = [1, 5, 1, 80, 3], [500, 260, 3, 400, 1000]
    s = Setup(news, lens, H, KH, D, gs, page, window)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("n,past", [(128, 0), (129, 0), (200, 333), (513, 64), (700, 0)])
@pytest.mark.parametrize("H,KH,D,gs,page", [(4, 2, 128, 128, 64), (8, 1, 128, 32, 16), (2, 2, 64, 64, 16),
                                            (3, 1, 96, 32, 32), (2, 1, 256, 128, 16)])
def test_prompts(gq4, n, past, H, KH, D, gs, page):
    s = Setup([n, 1], [past + n, 77], H, KH, D, gs, page)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("H,KH,D,gs,page", [(32, 8, 128, 128, 16), (32, 8, 128, 64, 64), (32, 4, 128, 32, 256),
                                            (64, 8, 64, 64, 16), (36, 12, 64, 32, 32), (35, 5, 96, 96, 16),
                                            (42, 6, 96, 32, 64), (16, 1, 128, 32, 16)])
@pytest.mark.parametrize("window", [0, 70])
def test_many_rows(gq4, H, KH, D, gs, page, window):
    """Enough query rows in all (2048) for the kernel of prompts, beside requests that are not its:
    whole tiles of 128 rows and 64 keys, one row and one key more, queries without keys."""
    news = [33, 64, 1, 130, 0, 9, 66, 40]
    lens = [33, 200, 65, 129, 5, 9, 64, 30]
    s = Setup(news, lens, H, KH, D, gs, page, window)
    assert s.T * H >= 2048
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("window", [33, 300])
def test_prompt_with_window(gq4, window):
    s = Setup([400, 300], [1000, 300], 4, 2, 128, 64, 16, window)
    s.check(s.run(gq4))


@pytest.mark.parametrize("length", [5000, 40003])
def test_long_contexts_split(gq4, length):
    s = Setup([1, 2], [length, 100], 8, 2, 128, 128, 64)
    s.check(s.run(gq4))


@pytest.mark.parametrize("H,KH,D,gs", [(8, 2, 64, 32), (2, 1, 128, 128)])
def test_more_requests_than_a_block_has_threads(gq4, H, KH, D, gs):
    """600 requests, idle and without keys among them, whose keys end anywhere in a stage; the
    first and the last are long, so that cuts fall inside and between requests."""
    g = I.rng(2202, H)
    news = g.integers(0, 4, 600).tolist()
    lens = [0 if g.random() < 0.05 else max(n, int(x)) for n, x in zip(news, g.integers(1, 260, 600))]
    news[0] = news[-1] = 1
    lens[0], lens[-1] = 2500, 1333
    s = Setup(news, lens, H, KH, D, gs, 16)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("H", [4, 16])
def test_queries_that_see_nothing(gq4, H):
    """seq_len < n: the first queries have no key (their rows are zeros); length 0."""
    s = Setup([5, 1, 200, 1], [2, 0, 30, 9], H, 2, 64, 32, 16)
    got = s.run(gq4)
    s.check(got)
    assert np.all(got[:3] == 0) and np.all(got[5] == 0) and np.all(got[6:6 + 170] == 0)


@pytest.mark.parametrize("H", [4, 16])
def test_sharp_and_flat_weights(gq4, H):
    """Queries that pick one key, and queries of zeros (the mean of the values)."""
    s = Setup([1, 1, 150], [600, 600, 700], H, 2, 128, 32, 16)
    s.q[0] *= 60
    s.q[1] = 0
    s.q[2:40] *= 30
    s.check(s.run(gq4))


def test_own_workspace_outlives_the_call_on_another_stream(gq4):
    """The workspace that a call allocates is not handed out again while its stream still uses it."""
    s = Setup([1, 1], [3000, 900], 8, 2, 128, 128, 16)
    clean = s.run(gq4)
    size = gq4.kv_attention_workspace_bytes(s.T, 8, 2, 128)
    args, q, out = s.dev(), dev(s.q), torch.full(s.q.shape, FILL, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    at = torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr()   # what the call will get
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    gq4.kv_attention(q, *args, scale=s.scale, max_query=1, max_len=3000, out=out, stream=side)
    again = torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr()
    assert again != at
    torch.cuda.synchronize()
    assert np.array_equal(host(out), clean)


def test_prompts_of_many_heads(gq4):
    """Queries without keys, that pick one key and that weigh all alike, scales over ten powers
    of two: 9000 and more query rows in all."""
    s = Setup([5, 1, 200, 1], [2, 0, 30, 9], 48, 4, 64, 32, 16)
    got = s.run(gq4)
    s.check(got)
    assert np.all(got[:3] == 0) and np.all(got[5] == 0) and np.all(got[6:6 + 170] == 0)
    for gs in (32, 128):
        s = Setup([1, 90, 150], [600, 600, 700], 40, 2, 128, gs, 16)
        s.q[0] *= 60
        s.q[1:30] = 0
        s.q[91:130] *= 30
        s.cache.sz[1][..., 0] *= np.exp2(np.random.default_rng(3).integers(-5, 6, s.cache.sz[1].shape[:-1]))
        s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("n,H", [(1, 4), (150, 4), (150, 16)])
def test_scales_of_unlike_size(gq4, n, H):
    """Value scales over ten powers of two, queries of very small and very large size."""
    s = Setup([n, n], [700, 800], H, 1, 128, 64, 16)
    g = I.rng(2201)
    for side, spread in ((0, 1.0), (1, 5.0)):
        sz = s.cache.sz[side]
        sz[..., 0] *= np.exp2(g.uniform(-spread, spread, sz.shape[:-1])).astype(np.float32)
    s.q[:n] *= 2.0 ** -100
    got = s.run(gq4)
    ref, tol = R.attention(s.q, s.starts, s.lens, s.table, s.cache, s.scale)
    live = 2 * n
    assert np.all(np.abs(got[:live] - ref[:live]) <= tol[:live])
    # queries and scale of opposite huge size give the same weights as plain ones
    s2 = Setup([n], [700], H, 1, 128, 64, 16)
    plain = s2.run(gq4)
    s2.q *= np.float32(2.0 ** 100)
    s2.scale *= 2.0 ** -100
    s2.check(s2.run(gq4))
    assert np.allclose(plain, s2.run(gq4), rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("n,heads,D", [(1, 1, 64), (140, 1, 64), (140, 4, 64), (140, 3, 128), (140, 4, 96)])
def test_non_finite_queries_and_keys_stay_apart(gq4, n, heads, D):
    """A NaN query spoils its own row; a NaN key or value only the rows that see it."""
    s = Setup([n, n], [200, 200], 4 * heads, 2 * heads, D, 32, 16)
    clean = s.run(gq4)
    q = s.q.copy()
    q[0, 1, 3] = np.nan
    q[0, 2, 5] = np.inf
    got = s.run(gq4, q=dev(q))
    assert np.isnan(got[0, 1]).all() and np.isnan(got[0, 2]).all()
    keep = np.ones(got.shape[:2], bool)
    keep[0, 1:3] = False
    assert np.array_equal(got[keep], clean[keep])
    # request 0's key 150 of kv head 1
    slot = s.table[0, 150 // 16], 150 % 16
    for side in range(2):
        kept = s.cache.sz[side][slot[0], 1, slot[1]].copy()
        s.cache.sz[side][slot[0], 1, slot[1]] = np.nan
        got = s.run(gq4)
        s.cache.sz[side][slot[0], 1, slot[1]] = kept
        sees = np.arange(n) + 200 - n >= 150
        assert np.isnan(got[:n][sees][:, 2:4]).all()
        assert np.array_equal(got[:n][~sees], clean[:n][~sees])
        others = [h for h in range(4 * heads) if h not in (2, 3)]
        assert np.array_equal(got[:n, others], clean[:n, others]) and np.array_equal(got[n:], clean[n:])


def test_strided_rows_and_workspace(gq4):
    s = Setup([1, 9, 30], [90, 40, 333], 6, 2, 64, 64, 16)
    H, KH, D = 6, 2, 64
    wide = torch.full((s.T, H + 2 * KH, D), 9.0, device="cuda")
    wide[:, :H] = dev(s.q)
    out = torch.full((s.T, H + 1, D), FILL, device="cuda")
    ws = torch.full((gq4.kv_attention_workspace_bytes(s.T, H, KH, D),), 255, dtype=torch.uint8, device="cuda")
    got = s.run(gq4, q=wide[:, :H], out=out[:, :H], workspace=ws)
    s.check(got)
    assert torch.all(out[:, H:] == FILL)


def test_bad_requests_are_refused(gq4):
    """Rows out of T, too many queries, too long, a page outside the pool: NaN rows and bit 8."""
    s = Setup([2, 3, 2, 2], [40, 50, 60, 70], 4, 2, 64, 32, 16, pad=0)
    clean = s.run(gq4)
    assert gq4.device_error(clear=True) == 0

    def spoiled(rows, **kw):
        got = s.run(gq4, **kw)
        assert gq4.device_error(clear=True) == 1 << 8
        keep = np.ones(s.T, bool)
        keep[rows] = False
        assert np.isnan(got[rows]).all()
        assert np.array_equal(got[keep], clean[keep])

    spoiled([2, 3, 4], max_query=2)
    spoiled([7, 8], max_len=65)
    args = s.dev()
    args[1] = dev(np.array([40, 50, 60, 10**6], np.int32))
    spoiled([7, 8], args=args, max_len=0)
    args[1] = dev(np.array([40, -1, 60, 70], np.int32))
    spoiled([2, 3, 4], args=args)
    args = s.dev()
    args[0] = dev(np.array([0, 2, 5, 7, 10**6], np.int32))     # the last request's rows pass T
    spoiled([7, 8], args=args, max_query=3)
    for page in (-1, 10**9):
        table = s.table.copy()
        table[1, 1] = page
        args = s.dev()
        args[2] = dev(table)
        spoiled([2, 3, 4], args=args)
    # rows of one request in another's order: the first begins before row 0
    args = s.dev()
    args[0] = dev(np.array([-4, 2, 5, 7, 9], np.int32))
    spoiled([0, 1], args=args, max_query=100)


@pytest.mark.parametrize("H", [2, 128])
def test_a_bad_page_spoils_only_the_rows_that_see_it(gq4, H):
    s = Setup([20], [40], H, 1, 64, 32, 16, pad=0)
    clean = s.run(gq4)
    s.table[0, 2] = -1          # keys 32..39: the last 8 queries
    got = s.run(gq4)
    assert gq4.device_error(clear=True) == 1 << 8
    assert np.array_equal(got[:12], clean[:12]) and np.isnan(got[12:]).all()


def test_same_bits_again_and_in_a_graph(gq4):
    s = Setup([1, 4, 1, 150], [3000, 900, 17, 400], 16, 4, 128, 64, 16)
    first = s.run(gq4)
    assert np.array_equal(first, s.run(gq4))
    args, q = s.dev(), dev(s.q)
    out = torch.full(s.q.shape, FILL, device="cuda")
    ws = torch.empty(gq4.kv_attention_workspace_bytes(s.T, 16, 4, 128), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):          # two graphs that share the workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                gq4.kv_attention(q, *args, scale=s.scale, max_query=150, max_len=3000, out=out, workspace=ws)
        graphs.append(g)
    for g in graphs * 2:
        out.fill_(FILL)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out), first)


def test_two_streams_at_once(gq4):
    a, b = Setup([1] * 8, [2000] * 8, 8, 2, 128, 128, 16), Setup([1, 200], [900, 500], 8, 2, 64, 32, 16)
    want = [s.run(gq4) for s in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    held = [(s.dev(), dev(s.q), torch.full(s.q.shape, FILL, device="cuda")) for s in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st, (args, q, out) in zip((a, b), streams, held):
            with torch.cuda.stream(st):
                gq4.kv_attention(q, *args, scale=s.scale, max_query=max(s.news), max_len=int(s.lens.max()), out=out)
    torch.cuda.synchronize()
    for w, (_, _, out) in zip(want, held):
        assert np.array_equal(host(out), w)


def test_cache_beyond_32_bits(gq4):
    """Pages whose codes start past 2^32 bytes: written, read back and attended to."""
    KH, D, gs, page, L = 8, 128, 128, 16, 50
    pages = (2**32) // (KH * page * D // 2) + 8
    c = gq4.kv_cache(pages, KH, page, D, gs)
    g = I.rng(2202)
    k, v = (g.standard_normal((L, KH, D)).astype(np.float32) for _ in range(2))
    table = np.array([[pages - 1, pages - 3, pages - 2, pages - 6]], np.int32)
    t = np.arange(L)
    slots = (table[0, t // page] * page + t % page).astype(np.int32)
    gq4.kv_append(dev(k), dev(v), dev(slots), *c, gs)
    kr, vr = gq4.kv_gather(dev(slots), *c, gs)
    q = g.standard_normal((1, 32, D)).astype(np.float32)
    out = gq4.kv_attention(dev(q), dev(np.array([0, 1], np.int32)), dev(np.array([L], np.int32)), dev(table), *c, gs,
                           scale=0.1, max_query=1)
    torch.cuda.synchronize()
    for x, r in ((k, kr), (v, vr)):
        codes, sz = R.quantise(x, gs)
        assert np.allclose(host(r), R.values(codes, sz), rtol=1e-6, atol=1e-6)
    kr, vr = host(kr).astype(np.float64), host(vr).astype(np.float64)
    for h in range(32):
        w = 0.1 * (kr[:, h // 4] @ q[0, h].astype(np.float64))
        w = np.exp(w - w.max())
        assert np.allclose(host(out)[0, h], w @ vr[:, h // 4] / w.sum(), rtol=1e-4, atol=1e-5)
    assert gq4.device_error(clear=True) == 0


def test_decode_loop(gq4):
    """A prompt and five steps of one layer's attention half: quad QKV product, norm and rotation,
    plan, append, attention, output projection, every link checked on what the GPU produced."""
    Hd, H, KH, D, gs, page, B = 512, 8, 2, 64, 64, 16, 3
    n0, n1, n2 = H * D, (H + KH) * D, (H + 2 * KH) * D
    wqkv, wo = I.quant_weights(Hd, n2, 64, 2300), I.quant_weights(n0, Hd, 64, 2301)
    g = I.rng(2302)
    gq, gk = (g.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))
    inv = (10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    pages, width = 40, 10
    cache = gq4.kv_cache(pages, KH, page, D, gs)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = dev(np.arange(pages, dtype=np.int32))
    count = dev(np.array([pages], np.int32))
    lens = dev(np.zeros(B, np.int32))
    written = [[[], []] for _ in range(B)]   # each request's k and v rows so far
    for step in range(6):
        news = [20, 1, 7] if step == 0 else [1, 1, 1]
        T = sum(news)
        x = I.activations(T, Hd, 2303, step)
        q, k, v, _ = gq4.quad_matvec(dev(x), *wdev(wqkv), 64, n0, n1, n2)
        C, S = oracle.matvec(x, wqkv.Bq, wqkv.scales, wqkv.zeros, Hd, n2, 64)
        tol = tol_fp32(S) if T < 16 else 2e-2 * S + 1e-6
        check_close("qkv", np.concatenate([host(t) for t in (q, k, v)], 1), C, tol)
        lens, starts, pos, slots, count = gq4.kv_plan(lens, dev(np.array(news, np.int32)), table, free, count, T, page)
        q3, k3, v3 = q.view(T, H, D), k.view(T, KH, D), v.view(T, KH, D)
        qr, kr = gq4.head_norm_rope(q3, k3, pos, dev(inv), q_gain=dev(gq), k_gain=dev(gk))
        gq4.kv_append(kr, v3, slots, *cache, gs)
        out = gq4.kv_attention(qr, starts, lens, table, *cache, gs, scale=D ** -0.5, max_query=max(news))
        o = gq4.matvec(out.view(T, n0), *wdev(wo), 64) if T <= 32 else None
        torch.cuda.synchronize()
        assert gq4.device_error() == 0
        y, size = R.norm_rope(host(q3), gq, 1e-6, host(pos), inv, False)
        assert np.all(np.abs(host(qr) - y) <= 16 * 2.0 ** -24 * size)
        y, size = R.norm_rope(host(k3), gk, 1e-6, host(pos), inv, False)
        assert np.all(np.abs(host(kr) - y) <= 16 * 2.0 ** -24 * size)
        row = 0
        for b, n in enumerate(news):
            for side, rows in enumerate((host(kr), host(v3))):
                written[b][side].extend(rows[row:row + n])
            kk, vv = (R.values(*R.quantise(np.stack(written[b][i]), gs)) for i in range(2))
            L = len(written[b][0])
            assert L == int(host(lens)[b])
            for j in range(n):
                seen = L - n + j + 1
                for h in range(H):
                    w = D ** -0.5 * (kk[:seen, h // (H // KH)] @ host(qr)[row + j, h].astype(np.float64))
                    w = np.exp(w - w.max())
                    ref = w @ vv[:seen, h // (H // KH)] / w.sum()
                    assert np.allclose(host(out)[row + j, h], ref, rtol=1e-4, atol=1e-4)
            row += n
        C, S = oracle.matvec(host(out).reshape(T, n0), wo.Bq, wo.scales, wo.zeros, n0, Hd, 64)
        check_close("o", host(o), C, tol_fp32(S) if T < 16 else 2e-2 * S + 1e-6)
