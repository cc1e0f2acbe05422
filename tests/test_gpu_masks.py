"""GPU tests of the attention over the paged 4-bit cache behind first tokens that stay visible and with drafted trees
(gq4_kv_attention_masked) against a float64 restatement (tests/mask_ref.py, whose bound tests/kv_ref.py derives)."""

import numpy as np
import pytest
import torch

from int4_group_quantized_quant_gb300 import inputs as I
from tests import kv_ref as R
from tests import mask_ref as M
from tests.gpu_util import dev, gq4_module, host, requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]

FILL = -1234.5


@pytest.fixture(scope="module")
def gq4():
    g = gq4_module()
    g.device_error(clear=True)
    return g


class Setup:
    """Requests over a pool with scattered pages; slots that no row sees hold NaN, pages without a seen slot lead nowhere.
    room: the length that the call is bounded by, and its tables wide enough for (trees of many heads go to the kernel of
    many rows by their rows times that)."""

    def __init__(self, news, lens, H, KH, D, gs, page, window=0, sinks=0, words=0, bits=None, pad=3, seed=0, room=None):
        g = I.rng(2400, sum(news), sum(lens), H, KH, D, gs, page, window, sinks, words, seed)
        self.news, self.lens = news, np.asarray(lens, np.int32)
        self.window, self.sinks, self.gs, self.scale = window, sinks, gs, 1.0 / np.sqrt(D)
        self.starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.T = int(self.starts[-1]) + pad
        self.bits = self.positions = None
        if words:
            parents = np.concatenate([M.random_parents(g, n) for n in news] + [np.zeros(pad, np.int32)])
            self.positions, self.bits, _ = M.tree(parents, self.starts, self.lens, words, window, sinks)
            if bits is not None:
                self.bits = bits(g, self.T, words)
        per = [(n + page - 1) // page for n in lens]
        pages = sum(per) + 3
        self.cache = R.Cache(g, pages, KH, page, D, gs)
        order = g.permutation(pages)
        self.room = room or (32768 if words and H >= 48 else int(max(lens)))
        self.table = np.full((len(lens), max(max(per) + 1, self.room // page)), -5, np.int32)
        used = np.zeros((pages, page), bool)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
            seen = self.sight(b).any(0) if news[b] else np.zeros(lens[b], bool)
            for t in np.nonzero(seen)[0]:
                used[self.table[b, t // page], t % page] = True
            for i in range(n):
                if window and not seen[i * page:(i + 1) * page].any() and (i + 1) * page <= lens[b] - news[b]:
                    self.table[b, i] = 10**9
        for side in range(2):
            self.cache.sz[side][np.broadcast_to(~used[:, None], self.cache.sz[side].shape[:3])] = np.nan
        self.q = g.standard_normal((self.T, H, D)).astype(np.float32)

    def sight(self, b):
        rows = slice(int(self.starts[b]), int(self.starts[b + 1]))
        return M.sight(self.news[b], int(self.lens[b]), self.window, self.sinks,
                       None if self.bits is None else self.bits[rows],
                       None if self.positions is None else self.positions[rows])

    def dev(self):
        return [dev(self.starts), dev(self.lens), dev(self.table), *[dev(a) for a in self.cache.arrays()], self.gs]

    def opts(self, **kw):
        o = dict(scale=self.scale, max_query=max(self.news), max_len=self.room, window=self.window,
                 sinks=self.sinks)
        if self.bits is not None:
            o["tree"] = dev(self.bits)
            if self.window:
                o["positions"] = dev(self.positions)
        o.update(kw)
        return o

    def run(self, gq4, q=None, args=None, **kw):
        out = torch.full(self.q.shape, FILL, device="cuda")
        opts = self.opts(out=out)
        opts.update(kw)
        gq4.kv_attention(dev(self.q) if q is None else q, *(args or self.dev()), **opts)
        torch.cuda.synchronize()
        return host(opts["out"])

    def ref(self):
        return M.attention(self.q, self.starts, self.lens, self.table, self.cache, self.scale, self.window, self.sinks,
                           self.bits, self.positions)

    def check(self, got):
        ref, tol = self.ref()
        live = int(self.starts[-1])
        assert np.all(got[live:] == FILL), "rows of no request changed"
        got, ref, tol = got[:live].astype(np.float64), ref[:live], tol[:live]
        assert np.all(np.isfinite(got))
        err = np.abs(got - ref)
        assert np.all(err <= tol), f"worst err/tol {float((err / np.maximum(tol, 1e-300)).max()):.3g}"
        assert np.linalg.norm(err) <= 1e-5 * np.linalg.norm(ref)


SHAPES = [
    # H, KH, D, gs, page
    (32, 8, 128, 128, 16), (4, 4, 64, 32, 16), (8, 1, 128, 32, 64), (6, 2, 96, 96, 32), (10, 2, 96, 32, 16),
    (7, 1, 256, 64, 128), (5, 1, 64, 64, 256), (3, 3, 256, 256, 16), (32, 2, 128, 64, 16), (40, 2, 64, 32, 64),
]
# rows for the kernel of prompts: 48 per kv head and 5120 in all
MANY = [(64, 8, 128, 128, 16), (64, 8, 128, 64, 64), (64, 4, 128, 32, 256), (64, 8, 64, 64, 16), (72, 12, 64, 32, 32),
        (70, 5, 96, 96, 16), (84, 6, 96, 32, 64), (48, 1, 128, 32, 16)]


@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 4), (50, 17), (33, 100), (200, 64), (70, 0), (5000, 4)])
@pytest.mark.parametrize("H,KH,D,gs,page", SHAPES)
def test_sinks(gq4, H, KH, D, gs, page, window, sinks):
    """Single tokens and few rows: sinks beyond the request, that touch the window, inside and at the edges of stages."""
    news = [1, 1, 5, 1, 1, 3, 1, 1, 2, 0, 1]
    lens = [1, 17, 260, 64, 300, 1000, 51, 500, 130, 40, 97]
    s = Setup(news, lens, H, KH, D, gs, page, window, sinks)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("window,sinks", [(20, 4), (70, 65), (130, 128), (64, 200), (300, 10)])
@pytest.mark.parametrize("H,KH,D,gs,page", MANY)
def test_sinks_of_many_rows(gq4, H, KH, D, gs, page, window, sinks):
    """Chunks of prompts for the kernel of many rows, beside requests that are not its."""
    news, lens = [130, 1, 66, 200], [530, 400, 66, 201]
    s = Setup(news, lens, H, KH, D, gs, page, window, sinks)
    assert s.T * H >= 5120
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (3, 0), (40, 4), (1000, 4)])
@pytest.mark.parametrize("H,KH,D,gs,page", SHAPES)
def test_trees(gq4, H, KH, D, gs, page, window, sinks):
    """Trees of one node to more than a word's, behind pasts that end anywhere in a stage; none at all; idle requests."""
    news = [1, 7, 15, 33, 2, 0, 40, 5, 31]
    lens = [1, 40, 15, 100, 66, 9, 300, 37, 95]
    s = Setup(news, lens, H, KH, D, gs, page, window, sinks, words=2)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (900, 4), (1000, 70)])
@pytest.mark.parametrize("H,KH,D,gs,page", MANY)
def test_trees_of_many_rows(gq4, H, KH, D, gs, page, window, sinks):
    """For the kernel of many rows: words in use and to spare, trees over several tiles of rows and of keys."""
    news, lens = [64, 33, 1, 100, 48], [64, 1333, 65, 1230, 47 + 128]
    s = Setup(news, lens, H, KH, D, gs, page, window, sinks, words=5)
    assert s.T * H * (window + sinks + 100 if window else s.room) >= 8 << 20
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("room", [0, 32768])
@pytest.mark.parametrize("requests", [1, 40, 255, 256, 257])
@pytest.mark.parametrize("H,KH,D,gs", [(8, 2, 128, 128), (14, 2, 64, 32), (5, 5, 96, 96)])
@pytest.mark.parametrize("words,window,sinks", [(1, 0, 0), (0, 100, 40), (1, 600, 4)])
def test_units_whole_and_cut(gq4, H, KH, D, gs, requests, room, words, window, sinks):
    """Bounds on the keys that let a unit of work be one block's, and ones that have it cut between blocks."""
    g = I.rng(2405, requests, H)
    news = [int(n) for n in g.integers(0, 4, requests)]
    news[0] = 9
    lens = [n + int(x) for n, x in zip(news, g.integers(0, 120, requests))]
    lens[0] = 1023
    s = Setup(news, lens, H, KH, D, gs, 16, window, sinks, words=words, room=room or max(1024, *lens))
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("H,KH", [(4, 2), (64, 2)])
def test_the_largest_trees(gq4, H, KH):
    s = Setup([256, 250], [256 + 19, 250 + 700], H, KH, 64, 32, 16, words=8)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("H,KH,D,gs", [(16, 2, 128, 128), (16, 2, 128, 64), (24, 2, 64, 32), (16, 1, 96, 96)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 20)])
def test_row_tiles_that_are_shared(gq4, H, KH, D, gs, window, sinks):
    """Trees behind long pasts: row tiles cut over two and over many CTAs, whole ones between them, small requests of the
    other kernel, and idle ones; lengths that are not those that the call is bounded by."""
    for news, lens in (([40], [6000]), ([33, 0, 40, 1, 64, 50, 20, 64], [5000, 9, 41, 700, 2000, 333, 1500, 64]),
                       ([64] * 20, [64 + 97 * i for i in range(20)])):
        s = Setup(news, lens, H, KH, D, gs, 16, window, sinks, words=2, room=32768)
        s.check(s.run(gq4))
        assert gq4.device_error() == 0


@pytest.mark.parametrize("gs", [128, 64])
def test_shared_row_tiles_of_unlike_size(gq4, gs):
    """Rows that their tile's pieces do not hold, in tiles that several CTAs share: each CTA sees a part of the keys."""
    s = Setup([64, 64], [5000, 3001], 8, 1, 128, gs, 16, words=2, room=32768)
    g = I.rng(2403)
    sz = s.cache.sz[1]
    sz[..., 0] *= np.exp2(g.uniform(-5, 5, sz.shape[:-1])).astype(np.float32)
    s.q[:128:7] *= np.float32(2.0 ** -60)
    big = 5000 - 64 + 3
    s.cache.sz[1][s.table[0, big // 16], :, big % 16, :, 0] *= np.float32(2.0 ** 20)
    s.check(s.run(gq4))
    first = s.run(gq4)
    assert np.array_equal(first, s.run(gq4)) and gq4.device_error() == 0


@pytest.mark.parametrize("H,KH,D,gs,page", [SHAPES[0], SHAPES[1], SHAPES[5], MANY[1], MANY[4]])
def test_any_bits(gq4, H, KH, D, gs, page):
    """Bits of no tree: later keys, not the row's own, none at all (with no past: a row of zeros), bits past the last key."""
    def bits(g, T, words):
        b = g.integers(0, 2**32, (T, words), dtype=np.uint32)
        b[::3] = 0
        b[1::5] = 0xffffffff
        return b
    news, lens = [40, 9, 3, 64, 50], [40, 77, 3, 200, 51]
    s = Setup(news, lens, H, KH, D, gs, page, words=2, bits=bits)
    got = s.run(gq4)
    s.check(got)
    assert np.all(got[0] == 0) and np.all(got[3] == 0)
    assert gq4.device_error() == 0


@pytest.mark.parametrize("H,KH", [(8, 2), (128, 2)])
def test_a_line_is_the_causal_rule(gq4, H, KH):
    """Bits of a line of drafts see what the causal call sees; first tokens within the window change nothing."""
    news, lens = [12, 30, 1], [200, 30, 90]
    s = Setup(news, lens, H, KH, 128, 128, 16)
    want = s.run(gq4)
    s.bits = np.zeros((s.T, 1), np.uint32)
    for b, n in enumerate(news):
        for j in range(n):
            s.bits[s.starts[b] + j] = 2 ** (j + 1) - 1
    s.check(s.run(gq4))
    s.bits, s.window, s.sinks = None, 500, 7
    got = s.run(gq4)
    live = int(s.starts[-1])
    _, tol = s.ref()
    assert np.all(np.abs(got[:live].astype(np.float64) - want[:live]) <= 2 * tol[:live])


def test_sinks_without_a_window_hide_nothing(gq4):
    s = Setup([1, 30], [700, 90], 8, 2, 128, 64, 16)
    want = s.run(gq4)
    s.sinks = 7
    assert np.array_equal(s.run(gq4), want)


@pytest.mark.parametrize("gs", [64, 32])
def test_trees_of_more_requests_than_a_block_has_threads(gq4, gs):
    """900 requests for the kernel of many rows: trees of one to three nodes of 64 heads, idle ones among them."""
    g = I.rng(2404, gs)
    news = g.integers(0, 4, 900).tolist()
    lens = [n + int(x) for n, x in zip(news, g.integers(0, 60, 900))]
    lens[450] += 3000
    s = Setup(news, lens, 64, 1, 64, gs, 16, words=1)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("gs", [128, 64])
def test_non_finite_queries_in_shared_row_tiles(gq4, gs):
    """A NaN or infinite query spoils its own row, in tiles that several CTAs share."""
    s = Setup([60], [7000], 16, 2, 128, gs, 16, words=2, room=32768)
    clean = s.run(gq4)
    s.check(clean)
    q = s.q.copy()
    q[3, 5, 7], q[40, 0, 100] = np.nan, np.inf
    got = s.run(gq4, q=dev(q))
    bad = np.zeros(got.shape[:2], bool)
    bad[3, 5] = bad[40, 0] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])
    assert gq4.device_error() == 0


def test_requests_that_share_rows_stay_in_bounds(gq4):
    """Requests over the same rows, between which one ends before it starts: more units than the call counts on."""
    s = Setup([64], [400], 64, 1, 64, 64, 16, words=2, pad=0)
    B = 301
    args = s.dev()
    args[0] = dev(np.array([0, 64] * (B // 2) + [0, 64], np.int32))
    args[1] = dev(np.full(B, 400, np.int32))
    args[2] = dev(np.repeat(s.table, B, 0))
    size = gq4.kv_attention_workspace_bytes(64, 64, 1, 64, tree=True)
    ws = torch.zeros(size + (1 << 20), dtype=torch.uint8, device="cuda")
    got = s.run(gq4, args=args, workspace=ws[:size])
    assert gq4.device_error(clear=True) == 1 << 8        # those that end before they start
    s.check(got)        # (how keys are split goes by the other requests: not to the bit)
    assert not ws[size:].any()


def test_a_bound_above_the_rows_of_the_call(gq4):
    """Fewer rows than max_query: the kernel and the workspace go by the rows."""
    s = Setup([2], [3000], 32, 8, 128, 128, 16, words=2, pad=0, room=1 << 20)
    size = gq4.kv_attention_workspace_bytes(2, 32, 8, 128, tree=True)
    ws = torch.zeros(size + (1 << 25), dtype=torch.uint8, device="cuda")
    s.check(s.run(gq4, max_query=64, workspace=ws[:size]))
    assert not ws[size:].any() and gq4.device_error() == 0
    for T, H, KH, D in ((16, 32, 8, 128), (64, 1, 1, 64), (1, 64, 1, 96), (8, 128, 8, 64)):     # the fewest rows of a tree call
        s = Setup([T], [3000], H, KH, D, D, 16, words=2, pad=0, room=1 << 20)
        size = gq4.kv_attention_workspace_bytes(T, H, KH, D, tree=True)
        ws = torch.zeros(size + (1 << 25), dtype=torch.uint8, device="cuda")
        s.check(s.run(gq4, workspace=ws[:size]))
        assert not ws[size:].any() and gq4.device_error() == 0


@pytest.mark.parametrize("H", [4, 64])
def test_queries_that_see_nothing(gq4, H):
    """seq_len < n with sinks and with bits; length 0."""
    s = Setup([5, 1, 120, 1], [2, 0, 30, 9], H, 2, 64, 32, 16, window=9, sinks=3)
    got = s.run(gq4)
    s.check(got)
    assert np.all(got[:3] == 0) and np.all(got[5] == 0)
    s = Setup([5, 1, 120, 1], [2, 0, 30, 9], H, 2, 64, 32, 16, words=4)
    s.check(s.run(gq4))


@pytest.mark.parametrize("H,KH,D,gs", [(8, 2, 64, 32), (2, 1, 128, 128)])
def test_more_requests_than_a_block_has_threads(gq4, H, KH, D, gs):
    g = I.rng(2401, H)
    news = g.integers(0, 9, 600).tolist()
    lens = [max(n, int(x)) for n, x in zip(news, g.integers(1, 260, 600))]
    lens[0], lens[-1] = 2500, 1333
    news[0] = news[-1] = 1
    s = Setup(news, lens, H, KH, D, gs, 16, words=1)
    s.check(s.run(gq4))
    s = Setup(news, lens, H, KH, D, gs, 16, window=60, sinks=4)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("window,sinks,words", [(4096, 4, 0), (0, 0, 1)])
def test_long_contexts_split(gq4, window, sinks, words):
    s = Setup([1, 2], [40003, 100], 8, 2, 128, 128, 64, window, sinks, words)
    s.check(s.run(gq4))


@pytest.mark.parametrize("H,KH,D,gs", [(8, 1, 128, 64), (64, 1, 128, 128), (64, 1, 64, 32), (64, 2, 96, 96)])
@pytest.mark.parametrize("window,sinks,words", [(90, 20, 0), (0, 0, 3), (60, 5, 3)])
def test_scales_of_unlike_size(gq4, H, KH, D, gs, window, sinks, words):
    """Value scales over ten powers of two, queries of very small size beside others, groups of equal values."""
    s = Setup([90, 80], [400, 333], H, KH, D, gs, 16, window, sinks, words)
    g = I.rng(2402)
    for side, spread in ((0, 1.0), (1, 5.0)):
        sz = s.cache.sz[side]
        sz[..., 0] *= np.exp2(g.uniform(-spread, spread, sz.shape[:-1])).astype(np.float32)
    s.q[:170:7] *= np.float32(2.0 ** -60)
    s.check(s.run(gq4))
    # one new key's value large, its neighbours' small: rows that do not see it keep their digits
    big = int(s.lens[0]) - s.news[0] + 3
    page, at = s.table[0, big // 16], big % 16
    s.cache.sz[1][page, :, at, :, 0] *= np.float32(2.0 ** 20)
    s.check(s.run(gq4))


@pytest.mark.parametrize("n,H", [(20, 4), (64, 96)])
def test_non_finite_keys_spoil_the_rows_that_see_them(gq4, n, H):
    for kw in (dict(words=2), dict(window=10, sinks=4)):
        s = Setup([n, n], [200, 200], H, 2, 64, 32, 16, **kw)
        clean = s.run(gq4)
        t = 2 if "sinks" in kw else 200 - n + 5
        slot = s.table[0, t // 16], t % 16
        sees = s.sight(0)[:, t]
        assert sees.any() and ("sinks" in kw or not sees.all())
        for side in range(2):
            kept = s.cache.sz[side][slot[0], 1, slot[1]].copy()
            s.cache.sz[side][slot[0], 1, slot[1]] = np.nan
            got = s.run(gq4)
            s.cache.sz[side][slot[0], 1, slot[1]] = kept
            half = slice(H // 2, H)
            assert np.isnan(got[:n][sees][:, half]).all()
            assert np.array_equal(got[:n][~sees], clean[:n][~sees])
            assert np.array_equal(got[:, :H // 2], clean[:, :H // 2]) and np.array_equal(got[n:], clean[n:])


@pytest.mark.parametrize("H", [4, 256])
def test_bad_pages_and_requests(gq4, H):
    """A page that only some rows see spoils those; one in the gap none; too many queries for the bits: NaN rows, bit 8."""
    s = Setup([20], [400], H, 2, 64, 32, 16, window=40, sinks=5, pad=0)
    clean = s.run(gq4)
    assert gq4.device_error(clear=True) == 0
    s.table[0, 5] = -1
    assert np.array_equal(s.run(gq4), clean) and gq4.device_error(clear=True) == 0
    kept = s.table[0, 24]
    s.table[0, 24] = 10**8                      # keys 384 .. 399: rows from 4 on
    got = s.run(gq4)
    assert gq4.device_error(clear=True) == 1 << 8
    assert np.array_equal(got[:4], clean[:4]) and np.isnan(got[4:]).all()
    s.table[0, 24] = kept
    s.table[0, 0] = -7
    got = s.run(gq4)
    assert gq4.device_error(clear=True) == 1 << 8 and np.isnan(got).all()
    s = Setup([20, 50, 3], [40, 70, 9], H, 2, 64, 32, 16, words=2, pad=0)
    clean = s.run(gq4)
    s.bits = s.bits[:, :1]
    got = s.run(gq4)
    assert gq4.device_error(clear=True) == 1 << 8
    assert np.isnan(got[20:70]).all() and np.isfinite(got[:20]).all() and np.array_equal(got[70:], clean[70:])


def test_positions_out_of_range_count_as_the_nearest(gq4):
    s = Setup([9, 70], [100, 300], 32, 2, 64, 32, 16, window=12, sinks=2, words=3)
    s.positions = np.where(np.arange(s.T) % 2, 10**9, -10**9).astype(np.int32)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("words,window,sinks", [(2, 0, 0), (0, 100, 4)])
def test_same_bits_again_and_in_a_graph(gq4, words, window, sinks):
    s = Setup([1, 4, 1, 50], [3000, 900, 17, 400], 128, 4, 128, 64, 16, window, sinks, words)
    first = s.run(gq4)
    assert np.array_equal(first, s.run(gq4))
    args, q = s.dev(), dev(s.q)
    out = torch.full(s.q.shape, FILL, device="cuda")
    ws = torch.empty(gq4.kv_attention_workspace_bytes(s.T, 128, 4, 128, tree=True), dtype=torch.uint8, device="cuda")
    opts = s.opts(out=out, workspace=ws)
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):          # two graphs that share the workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                gq4.kv_attention(q, *args, **opts)
        graphs.append(g)
    for g in graphs * 2:
        out.fill_(FILL)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out), first)


def test_two_streams_at_once(gq4):
    a = Setup([9] * 8, [2000] * 8, 8, 2, 128, 128, 16, words=1)
    b = Setup([1, 200], [900, 500], 32, 2, 64, 32, 16, window=60, sinks=4)
    want = [s.run(gq4) for s in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    held = [(s.dev(), dev(s.q), s.opts(out=torch.full(s.q.shape, FILL, device="cuda"))) for s in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (args, q, opts) in zip(streams, held):
            with torch.cuda.stream(st):
                gq4.kv_attention(q, *args, **opts)
    torch.cuda.synchronize()
    for w, (_, _, opts) in zip(want, held):
        assert np.array_equal(host(opts["out"]), w)


def test_strided_rows_and_workspace(gq4):
    s = Setup([1, 9, 30], [90, 40, 333], 6, 2, 64, 64, 16, window=50, sinks=3, words=1)
    H, KH, D = 6, 2, 64
    wide = torch.full((s.T, H + 2 * KH, D), 9.0, device="cuda")
    wide[:, :H] = dev(s.q)
    out = torch.full((s.T, H + 1, D), FILL, device="cuda")
    ws = torch.full((gq4.kv_attention_workspace_bytes(s.T, H, KH, D, tree=True),), 255, dtype=torch.uint8, device="cuda")
    s.check(s.run(gq4, q=wide[:, :H], out=out[:, :H], workspace=ws))
    assert torch.all(out[:, H:] == FILL)


def test_the_binding_refuses(gq4):
    s = Setup([3], [40], 4, 2, 64, 32, 16, words=1)
    with pytest.raises(ValueError, match="positions"):
        s.run(gq4, window=5)
    with pytest.raises(ValueError, match="tree"):
        s.run(gq4, tree=dev(s.bits[:-1]))
    with pytest.raises(ValueError, match="tree's"):
        s.run(gq4, tree=None, positions=dev(s.positions))
    with pytest.raises(gq4.GQ4Error):
        s.run(gq4, sinks=-1)
    with pytest.raises(gq4.GQ4Error):
        s.run(gq4, tree=torch.zeros(s.T, 9, dtype=torch.int32, device="cuda"))
