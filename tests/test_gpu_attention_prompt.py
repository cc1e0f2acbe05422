"""GPU tests of gq4_kv_attention's kernel for requests with many query rows
(prompts and chunks), and of both kernels on caches and queries of unlike
sizes, against the float64 restatement of tests/kv_ref.py.

Every case that is meant for the prompt kernel states so by ``prompt(...)``,
which restates the dispatch rule: at least 48 query rows per kv head in some
request, 5120 in all, heads of at most 128 values."""

import numpy as np
import pytest
import torch

from int4_group_quantized_quant_gb300 import inputs as I
from tests import kv_ref as R
from tests.gpu_util import dev, gq4_module, host, requires_cuda
from tests.test_gpu_attention import FILL, Setup

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def gq4():
    g = gq4_module()
    g.device_error(clear=True)
    return g


def prompt(news, lens, H, KH, D, gs, page, window=0, pad=3, seed=0):
    """A Setup whose requests of 48 query rows per kv head and more run on the prompt kernel."""
    s = Setup(news, lens, H, KH, D, gs, page, window, pad, seed)
    assert max(news) * (H // KH) >= 48 and s.T * H >= 5120 and D <= 128
    return s


def few(news, lens, H, KH, D, gs, page, window=0, pad=3, seed=0):
    """A Setup that runs on the kernel of few query rows."""
    s = Setup(news, lens, H, KH, D, gs, page, window, pad, seed)
    assert max(news) * (H // KH) < 48 or s.T * H < 5120 or D > 128
    return s


def close(got, s, shrink=1.0):
    """Within the derived bound (times shrink) everywhere; returns the worst share of it."""
    ref, tol = R.attention(s.q, s.starts, s.lens, s.table, s.cache, s.scale, s.window)
    live = int(s.starts[-1])
    got, ref, tol = got[:live].astype(np.float64), ref[:live], shrink * tol[:live]
    assert np.all(np.isfinite(got))
    err = np.abs(got - ref)
    assert np.all(err <= tol), f"worst err/tol {float((err / np.maximum(tol, 1e-300)).max()):.3g}"


# H, KH, D, gs: one group and several, padded heads, groups of query heads of any size
FORMS = [(24, 6, 128, 128), (24, 6, 128, 64), (24, 3, 128, 32), (20, 4, 96, 96), (24, 8, 96, 32), (32, 4, 64, 64),
         (20, 20, 64, 32)]


# ---------------------------------------------------------------------------
# The prompt kernel: masks, rows, what is not finite, pages, repetition
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("window", [1, 16, 33, 64, 300])
@pytest.mark.parametrize("H,KH,D,gs", FORMS)
def test_windows(gq4, H, KH, D, gs, window):
    s = prompt([140, 60, 1, 90], [500, 60, 70, 333], H, KH, D, gs, 32, window)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("H,KH,D,gs", FORMS)
def test_what_is_not_finite_stays_apart(gq4, H, KH, D, gs):
    """A NaN or infinite query spoils its own row; a NaN key or value only the rows that see it."""
    n, L, R_ = 140, 200, H // KH
    s = prompt([n, n], [L, L], H, KH, D, gs, 16)
    clean = s.run(gq4)
    q = s.q.copy()
    q[0, 1, 3] = np.nan
    q[n - 1, 2, 5] = np.inf
    q[5, 3, D - 1] = -np.inf
    got = s.run(gq4, q=dev(q))
    keep = np.ones(got.shape[:2], bool)
    for row, h in ((0, 1), (n - 1, 2), (5, 3)):
        assert np.isnan(got[row, h]).all()
        keep[row, h] = False
    assert np.array_equal(got[keep], clean[keep])
    slot = s.table[0, 150 // 16], 150 % 16            # request 0's key 150 of kv head 1
    sees = np.arange(n) + L - n >= 150
    mine = list(range(R_, 2 * R_))
    others = [h for h in range(H) if h not in mine]
    for side in range(2):
        kept = s.cache.sz[side][slot[0], 1, slot[1]].copy()
        s.cache.sz[side][slot[0], 1, slot[1]] = np.nan
        got = s.run(gq4)
        s.cache.sz[side][slot[0], 1, slot[1]] = kept
        assert np.isnan(got[:n][sees][:, mine]).all()
        assert np.array_equal(got[:n][~sees], clean[:n][~sees])
        assert np.array_equal(got[:n, others], clean[:n, others]) and np.array_equal(got[n:], clean[n:])
    assert gq4.device_error() == 0


@pytest.mark.parametrize("H,KH,D,gs", [(256, 1, 64, 32), (256, 2, 64, 64), (256, 4, 128, 128), (260, 5, 96, 32)])
@pytest.mark.parametrize("page", [-1, 10**9])
def test_a_bad_page_spoils_only_the_rows_that_see_it(gq4, H, KH, D, gs, page):
    s = prompt([20], [40], H, KH, D, gs, 16, pad=0)
    clean = s.run(gq4)
    s.table[0, 2] = page        # keys 32..39: the last 8 queries
    got = s.run(gq4)
    assert gq4.device_error(clear=True) == 1 << 8
    assert np.array_equal(got[:12], clean[:12]) and np.isnan(got[12:]).all()


@pytest.mark.parametrize("H,KH,D,gs", FORMS)
def test_same_bits_again_and_in_graphs(gq4, H, KH, D, gs):
    """Twice, and in two graphs that share the workspace, replayed in turn; NaN in the workspace."""
    s = prompt([1, 4, 130, 150], [900, 300, 200, 400], H, KH, D, gs, 16)
    first = s.run(gq4)
    assert np.array_equal(first, s.run(gq4))
    args, q = s.dev(), dev(s.q)
    out = torch.full(s.q.shape, FILL, device="cuda")
    ws = torch.full((gq4.kv_attention_workspace_bytes(s.T, H, KH, D),), 255, dtype=torch.uint8, device="cuda")
    side, graphs = torch.cuda.Stream(), []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                gq4.kv_attention(q, *args, scale=s.scale, max_query=150, max_len=900, out=out, workspace=ws)
        graphs.append(g)
    for g in graphs * 2:
        out.fill_(FILL)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out), first)


@pytest.mark.parametrize("H,KH,D,gs", [(24, 6, 128, 128), (24, 6, 128, 32), (24, 8, 96, 96)])
def test_strided_rows(gq4, H, KH, D, gs):
    """q as columns of the fused QKV product, out as columns of a wider matrix."""
    s = prompt([150, 77], [150, 333], H, KH, D, gs, 16)
    wide = torch.full((s.T, H + 2 * KH, D), 9.0, device="cuda")
    wide[:, :H] = dev(s.q)
    out = torch.full((s.T, H + 1, D), FILL, device="cuda")
    got = s.run(gq4, q=wide[:, :H], out=out[:, :H])
    s.check(got)
    assert torch.all(out[:, H:] == FILL)


def test_two_streams_at_once(gq4):
    a, b = prompt([150, 99], [500, 99], 24, 6, 128, 128, 16), prompt([1, 200], [900, 500], 32, 8, 64, 32, 16)
    want = [s.run(gq4) for s in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    held = [(s.dev(), dev(s.q), torch.full(s.q.shape, FILL, device="cuda")) for s in (a, b)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, st, (args, q, out) in zip((a, b), streams, held):
            with torch.cuda.stream(st):
                gq4.kv_attention(q, *args, scale=s.scale, max_query=max(s.news), max_len=int(s.lens.max()), out=out)
    torch.cuda.synchronize()
    for w, (_, _, out) in zip(want, held):
        assert np.array_equal(host(out), w)


@pytest.mark.parametrize("H,KH,D,gs", FORMS)
def test_sizes_of_queries_and_scales(gq4, H, KH, D, gs):
    """Value scales over ten powers of two, a request of queries 2^-100 of the other's; queries and
    scale of opposite huge size."""
    n = 130
    s = prompt([n, n], [300, 400], H, KH, D, gs, 16)
    g = I.rng(2210)
    for side, spread in ((0, 1.0), (1, 5.0)):
        sz = s.cache.sz[side]
        sz[..., 0] *= np.exp2(g.uniform(-spread, spread, sz.shape[:-1])).astype(np.float32)
    s.q[:n] *= 2.0 ** -100
    close(s.run(gq4), s)
    s = prompt([2 * n], [400], H, KH, D, gs, 16)
    s.q *= np.float32(2.0 ** 100)
    s.scale *= 2.0 ** -100
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


# ---------------------------------------------------------------------------
# Values, keys and queries of unlike size, on both kernels
# ---------------------------------------------------------------------------

BOTH = [(prompt, [200, 1, 64], [300, 77, 64], *f) for f in FORMS] + \
       [(few, [5, 1, 3], [300, 77, 3], *f) for f in [*FORMS, (8, 8, 128, 128), (4, 4, 256, 64), (12, 2, 256, 256)]]


def name_of(x):
    return x.__name__ if callable(x) else None


@pytest.mark.parametrize("make,news,lens,H,KH,D,gs", BOTH, ids=name_of)
def test_rows_of_scale_zero(gq4, make, news, lens, H, KH, D, gs):
    """Value and key rows whose scales are 0 (an unwritten slot of a zeroed pool) count as zeros."""
    s = make(news, lens, H, KH, D, gs, 16)
    g = I.rng(2211, H, D, gs)
    for side in range(2):
        live = ~np.isnan(s.cache.sz[side][..., 0, 0])
        s.cache.sz[side][live & (g.random(live.shape) < 0.3)] = 0.0
    s.check(s.run(gq4))
    for side in range(2):
        s.cache.sz[side][~np.isnan(s.cache.sz[side])] = 0.0
    got = s.run(gq4)
    assert np.all(got[:int(s.starts[-1])] == 0.0)
    assert gq4.device_error() == 0


@pytest.mark.parametrize("make,news,lens,H,KH,D,gs", BOTH, ids=name_of)
@pytest.mark.parametrize("power", [16, 24, 40, 100])
def test_scores_of_any_size(gq4, make, news, lens, H, KH, D, gs, power):
    """Queries so large that the exponents pass 2^24: an output is still a mean of the values with
    weights that sum to 1, and the top key's value where no error of the exponents can decide."""
    s = make(news, lens, H, KH, D, gs, 16)
    s.q *= np.float32(2.0 ** power)
    got = s.run(gq4).astype(np.float64)
    R_ = H // KH
    sure = 0
    for b, (n, L) in enumerate(zip(news, lens)):
        t = np.arange(L)
        slots = s.table[b, t // 16].astype(np.int64) * 16 + t % 16
        seen = t[None] <= (L - n + np.arange(n))[:, None]
        for h in range(H):
            k, v = (s.cache.rows(side, h // R_, slots) for side in range(2))
            x = s.q[s.starts[b]:s.starts[b] + n, h].astype(np.float64)
            w = np.where(seen, s.scale * (x @ k.T), -np.inf)
            # twice the restated bound's error of an exponent, from a looser A: |code - z| <= 9
            e = 2 * s.scale * np.abs(x).sum(-1) * 0.3 * 24 * (D / 8 + 9) * 2.0 ** -23
            out = got[s.starts[b]:s.starts[b] + n, h]
            vmax = np.abs(v).max()
            assert np.all(np.abs(out) <= vmax * 1.001)
            top = np.sort(w, -1)[:, -2:] if L > 1 else np.stack([np.full(n, -np.inf), w[:, 0]], -1)
            one = top[:, 1] - top[:, 0] > 2 * e + 20
            sure += one.sum()
            # 2^-20 of the rest's weight and the bound's 16 units on terms of 17 scales of 0.3
            assert np.all(np.abs(out[one] - v[np.argmax(w[one], -1)]) <= L * np.exp(-20.0) * vmax + 16 * 2.0 ** -23 * 5.1)
    assert sure > 0
    assert gq4.device_error() == 0


@pytest.mark.parametrize("make,news,lens,H,KH,D,gs", BOTH, ids=name_of)
@pytest.mark.parametrize("low,high,by", [(0, 40, 0), (0, 13, 0), (-60, 40, 0), (-70, -30, 50), (60, 120, -80)])
def test_queries_of_unlike_size(gq4, make, news, lens, H, KH, D, gs, low, high, by):
    """Rows of one request spread over many powers of two (the scale taken by 2^by): every row is
    held to the bound of its own size, whatever rows stand beside it."""
    s = make(news, lens, H, KH, D, gs, 16)
    g = I.rng(2212, H, D, gs)
    size = g.integers(low, high + 1, s.q.shape[:2])
    size[::3] = min(max(-by, low), high)         # a third of the tokens: weights of ordinary spread
    s.q *= np.exp2(size).astype(np.float32)[..., None]
    s.q[7 % len(s.q), 1] = 0.0
    s.scale = np.ldexp(s.scale, by)
    close(s.run(gq4), s)
    assert gq4.device_error() == 0


@pytest.mark.parametrize("make,news,lens,H,KH,D,gs", BOTH, ids=name_of)
@pytest.mark.parametrize("power", [20, 40, 90])
@pytest.mark.parametrize("window", [0, 40])
def test_unseen_values_take_no_digits(gq4, make, news, lens, H, KH, D, gs, power, window):
    """Values 2^power of the others' size at a request's last keys, and before the window's first:
    the rows that do not see them are held to the bound of what they see."""
    s = make(news, lens, H, KH, D, gs, 16, window)
    for b, n in enumerate(lens):
        at = [n - 1, n - 30] if news[b] > 40 else [n - 1]
        if window:
            at.append(max(0, n - news[b] + 1 - window))     # the first query's first key
        for t in at:
            s.cache.sz[1][s.table[b, t // 16], :, t % 16, :, 0] *= np.float32(2.0 ** power)
    close(s.run(gq4), s)
    assert gq4.device_error() == 0


@pytest.mark.parametrize("H,KH,D,gs", FORMS)
@pytest.mark.parametrize("jump", [20, 30, 45, 100])
def test_a_reference_that_jumps_inside_a_tile(gq4, H, KH, D, gs, jump):
    """47 keys just below 2^4 of the first ones' weight, then one of 2^jump: what was summed before
    shrinks by the whole jump.  The last key's value is 0 and its weight is all but everything, so
    the result is below 48 2^(4 - jump) of the others' values (1) and its error below 16 2^-23 of
    them, whatever the error of the exponents is (the bound's own term for them does not apply)."""
    s = prompt([260], [330], H, KH, D, gs, 16)
    t = np.arange(330)
    log2w = np.where(t < 16, 0.0, np.where(t < 63, 3.875, np.where(t == 63, 3.875 + jump, -40.0)))
    s.q[:] = 1.0
    slots = s.table[0, t // 16], t % 16
    # code 1, zero 0 in every key: w = scale D s
    s.cache.codes[0][:] = 1
    sk = (log2w / (s.scale * D * np.log2(np.e))).astype(np.float32)
    for i in range(330):
        pg, at = slots[0][i], slots[1][i]
        s.cache.sz[0][pg, :, at, :] = (sk[i], 0.0)
        s.cache.sz[1][pg, :, at, :] = (1.0 / 16, 0.0)
        s.cache.codes[1][pg, :, at] = 0 if i == 63 else 15
    got = s.run(gq4)[:260].astype(np.float64)
    ref, _ = R.attention(s.q, s.starts, s.lens, s.table, s.cache, s.scale)
    assert np.all(np.abs(got - ref[:260]) <= 16 * 2.0 ** -23 + 48 * 2.0 ** (4 - jump) * 2.0 ** -15)


@pytest.mark.parametrize("make,news,lens,H,KH,D,gs", BOTH, ids=name_of)
@pytest.mark.parametrize("size", [1e-3, 1e-6, 1e3])
def test_groups_of_one_value(gq4, make, news, lens, H, KH, D, gs, size):
    """A group of equal values has scale 1, codes 0 and the value in its zero (the quantiser's rule);
    a row of zeros among them.  Errors are held to the values' size, not to the scale's: the bound
    with s (code + |z|), at most `top` here, in the place of s (8 + |z - 8|), 16 at least where s = 1."""
    s = make(news, lens, H, KH, D, gs, 16)
    g = I.rng(2213, H, D, gs)
    sz = s.cache.sz[1]
    live = ~np.isnan(sz[..., 0])                               # [page, head, slot, group]
    ordinary = np.where(live[..., None], sz, 0.0)
    const = live & (g.random(live.shape) < 0.5)
    for b, n in enumerate(lens):                               # every row sees one: the first key
        if n:
            const[s.table[b, 0], :, 0] = True
    lo = (size * g.uniform(-1, 1, live.shape)).astype(np.float32)
    lo[g.random(live.shape) < 0.2] = 0.0
    sz[..., 0] = np.where(const, 1.0, sz[..., 0] * np.float32(size))
    sz[..., 1] = np.where(const, -lo, sz[..., 1])
    s.cache.codes[1][np.repeat(const, gs, -1)] = 0
    top = max(float(np.abs(lo).max()), size * float((ordinary[..., 0] * (15 + ordinary[..., 1])).max()))
    # in the restated bound every row's vmax is that of some group with s = 1: 8 + |z - 8|
    least = 16.0 if size < 1 else 8.0
    close(s.run(gq4), s, min(1.0, top / least))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("make,news,lens,H,KH,D,gs", BOTH, ids=name_of)
def test_keys_of_one_value(gq4, make, news, lens, H, KH, D, gs):
    """The same among the keys, under queries that make up for their size (the restated bound holds
    as it is: it counts a key's codes and zero)."""
    s = make(news, lens, H, KH, D, gs, 16)
    g = I.rng(2214, H, D, gs)
    sz = s.cache.sz[0]
    live = ~np.isnan(sz[..., 0])
    const = live & (g.random(live.shape) < 0.5)
    lo = (1e-3 * g.uniform(-1, 1, live.shape)).astype(np.float32)
    sz[..., 0] = np.where(const, 1.0, sz[..., 0] * np.float32(1e-3))
    sz[..., 1] = np.where(const, -lo, sz[..., 1])
    s.cache.codes[0][np.repeat(const, gs, -1)] = 0
    s.q *= np.float32(1e3)
    s.check(s.run(gq4))
    assert gq4.device_error() == 0


@pytest.mark.parametrize("make,news,lens,H,KH,D,gs", [BOTH[0], BOTH[2], BOTH[len(FORMS)]], ids=name_of)
def test_rows_that_end_before_they_start(gq4, make, news, lens, H, KH, D, gs):
    """query_start that decreases: that request has no rows and bit 8 is set; the others are served."""
    s = make(news, lens, H, KH, D, gs, 16)
    assert gq4.device_error(clear=True) == 0
    args = s.dev()
    args[0] = dev(np.array([0, news[0], news[0] - 2, s.starts[3]], np.int32))
    got = s.run(gq4, args=args, max_query=max(news) + 4)
    assert gq4.device_error(clear=True) == 1 << 8
    # (how keys are split depends on the other requests, so last bits may differ: the bound holds)
    ref, tol = R.attention(s.q, s.starts, s.lens, s.table, s.cache, s.scale)
    mine = slice(0, news[0] - 2)
    assert np.all(np.abs(got[mine] - ref[mine]) <= tol[mine])
    assert np.all(got[s.starts[3]:] == FILL)


@pytest.mark.parametrize("make,news,lens,H,KH,D,gs",
                         [c for c in BOTH if c[5] > c[6]], ids=name_of)
def test_a_value_group_that_is_not_finite(gq4, make, news, lens, H, KH, D, gs):
    """A NaN scale of one group of one value row: the rows that see it are NaN in that group's
    columns at least (all of theirs in the prompt kernel), the others as they were."""
    s = make(news, lens, H, KH, D, gs, 16)
    clean = s.run(gq4)
    ref, tol = R.attention(s.q, s.starts, s.lens, s.table, s.cache, s.scale)
    R_, n, L, at = H // KH, news[0], lens[0], lens[0] - 2
    sees = np.arange(n) + L - n >= at
    for group in range(D // gs):
        kept = s.cache.sz[1][s.table[0, at // 16], 0, at % 16, group].copy()
        s.cache.sz[1][s.table[0, at // 16], 0, at % 16, group] = np.nan
        got = s.run(gq4)
        s.cache.sz[1][s.table[0, at // 16], 0, at % 16, group] = kept
        cols = np.zeros(D, bool)
        cols[group * gs:(group + 1) * gs] = True
        mine = got[:n][sees][:, :R_]
        assert np.isnan(mine[..., cols]).all()
        if make is few:
            err = np.abs(mine - ref[:n][sees][:, :R_])[..., ~cols]
            assert np.all(err <= tol[:n][sees][:, :R_][..., ~cols])
        else:
            assert np.isnan(mine).all()
        assert np.array_equal(got[:n][~sees], clean[:n][~sees]) and np.array_equal(got[n:], clean[n:])
        assert np.array_equal(got[:n][sees][:, R_:], clean[:n][sees][:, R_:])
    assert gq4.device_error() == 0


@pytest.mark.parametrize("n,B,idle", [(12, 40, 0), (12, 17, 300), (13, 25, 900), (33, 30, 5)])
def test_requests_of_the_fewest_rows(gq4, n, B, idle):
    """Requests of 48 query rows per kv head, the fewest of this kernel, and a little more, between
    others without queries or with one: the launch has a tile for each, and a mark for each tile."""
    g = I.rng(2215, n, B, idle)
    news = [n] * B + g.integers(0, 2, idle).tolist()
    lens = [n + int(x) for x in g.integers(0, 60, B)] + [1 + int(x) for x in g.integers(0, 30, idle)]
    order = g.permutation(B + idle)
    news, lens = [news[i] for i in order], [lens[i] for i in order]
    for H, KH, D, gs in ((32, 8, 64, 64), (32, 8, 64, 32)):
        s = prompt(news, lens, H, KH, D, gs, 16)
        s.check(s.run(gq4))
        s.q *= np.exp2(g.integers(-20, 20, s.q.shape[:2])).astype(np.float32)[..., None]
        close(s.run(gq4), s)
    assert gq4.device_error() == 0
