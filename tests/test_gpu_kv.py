"""GPU tests of the per-head norm with rotation (gq4_head_norm_rope), the paged
4-bit cache's writer and reader (gq4_kv_append, gq4_kv_gather) and a step's
book-keeping (gq4_kv_plan).

Bars: the cache's codes, scales and zeros and everything the plan writes are
equal bit for bit; the rotation is held to 16 units of 2^-24 of |y_a| + |y_b|
(one rounding each for the mean's terms in pairs, the root, the quotient, two
products, sine and cosine within 2 units each of 2^-24 and their angle's
rounding 2^-23 |a|, and the last two products and the sum).
"""

import numpy as np
import pytest
import torch

from int4_group_quantized_quant_gb300 import inputs as I
from tests import kv_ref as R
from tests.gpu_util import Guarded, dev, gq4_module, host, requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def gq4():
    g = gq4_module()
    g.device_error(clear=True)
    return g


# ---------------------------------------------------------------------------
# Norm and rotation
# ---------------------------------------------------------------------------

ROPE_CASES = [
    # T, H, KH, D, rot, interleaved, norm
    (1, 32, 8, 128, 128, False, True),
    (1, 1, 0, 64, 64, True, False),
    (3, 0, 5, 96, 48, False, True),
    (7, 5, 1, 256, 128, True, True),
    (2, 3, 3, 8, 8, False, True),
    (5, 9, 2, 40, 24, False, True),      # rows that do not fill their lanes
    (4, 2, 2, 512, 512, False, True),
    (4, 2, 2, 200, 0, False, True),      # norm only
    (130, 16, 4, 128, 32, True, False),  # rotation only
    (513, 14, 2, 64, 64, False, True),
]


def rope_inputs(T, H, KH, D, rot, seed, top=100000):
    g = I.rng(2100, T, H, KH, D, rot, seed)
    q = g.standard_normal((T, H, D)).astype(np.float32)
    k = g.standard_normal((T, KH, D)).astype(np.float32)
    pos = g.integers(0, top, T, dtype=np.int64).astype(np.int32)
    inv = (10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)
    gq, gk = (g.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))
    return q, k, pos, inv, gq, gk


def check_rope(got, x, gain, eps, pos, inv, interleaved):
    ref, size = R.norm_rope(x, gain, eps, pos, inv, interleaved)
    err = np.abs(host(got).astype(np.float64) - ref)
    bound = 16 * 2.0 ** -24 * size + 1e-30
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("T,H,KH,D,rot,interleaved,norm", ROPE_CASES)
def test_rope(gq4, T, H, KH, D, rot, interleaved, norm):
    q, k, pos, inv, gq, gk = rope_inputs(T, H, KH, D, rot, 0)
    qo, ko = Guarded((T, H, D)), Guarded((T, KH, D))
    gq4.head_norm_rope(dev(q) if H else None, dev(k) if KH else None, dev(pos) if rot else None,
                       dev(inv) if rot else None, q_gain=dev(gq) if norm and H else None,
                       k_gain=dev(gk) if norm and KH else None, eps=1e-5, interleaved=interleaved,
                       q_out=qo.t if H else None, k_out=ko.t if KH else None)
    torch.cuda.synchronize()
    inv = inv if rot else None
    if H:
        qo.check()
        check_rope(qo.t, q, gq if norm else None, 1e-5, pos, inv, interleaved)
    if KH:
        ko.check()
        check_rope(ko.t, k, gk if norm else None, 1e-5, pos, inv, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_in_place_in_a_fused_row(gq4, interleaved):
    """q and k are column blocks of one matrix and are rotated where they stand; v stays."""
    T, H, KH, D = 37, 6, 2, 128
    q, k, pos, inv, gq, gk = rope_inputs(T, H, KH, D, D, 1)
    v = I.rng(2101).standard_normal((T, KH, D)).astype(np.float32)
    fused = dev(np.concatenate([q, k, v], 1))
    a, b = fused[:, :H], fused[:, H:H + KH]
    gq4.head_norm_rope(a, b, dev(pos), dev(inv), q_gain=dev(gq), q_out=a, k_out=b, interleaved=interleaved)
    torch.cuda.synchronize()
    check_rope(a, q, gq, 1e-6, pos, inv, interleaved)
    check_rope(b, k, None, 1e-6, pos, inv, interleaved)
    assert np.array_equal(host(fused[:, H + KH:]), v)


def test_rope_far_positions(gq4):
    """Angles up to 2^31 lose nothing; zero and negative positions turn the right way."""
    T, H, D = 64, 2, 128
    q, _, _, inv, _, _ = rope_inputs(T, H, 0, D, D, 2)
    pos = I.rng(2102).integers(2**31 - 4096, 2**31, T, dtype=np.int64).astype(np.int32)
    pos[:4] = [0, -1, 2**31 - 1, -2**31]
    out, _ = gq4.head_norm_rope(dev(q), None, dev(pos), dev(inv))
    torch.cuda.synchronize()
    check_rope(out, q, None, 1e-6, pos, inv, False)


def test_rope_non_finite_rows_stay_apart(gq4):
    T, H, D = 3, 4, 64
    q, _, pos, inv, gq, _ = rope_inputs(T, H, 0, D, D, 3)
    bad = q.copy()
    bad[1, 2, 5] = np.nan
    bad[2, 0, 7] = np.inf
    clean, _ = gq4.head_norm_rope(dev(q), None, dev(pos), dev(inv), q_gain=dev(gq))
    out, _ = gq4.head_norm_rope(dev(bad), None, dev(pos), dev(inv), q_gain=dev(gq))
    torch.cuda.synchronize()
    out, clean = host(out), host(clean)
    assert np.isnan(out[1, 2]).all()
    assert not np.isfinite(out[2, 0, 7])
    keep = np.ones((T, H), bool)
    keep[1, 2] = keep[2, 0] = False
    assert np.array_equal(out[keep], clean[keep])


# ---------------------------------------------------------------------------
# Cache: writer and reader
# ---------------------------------------------------------------------------

CACHE_CASES = [
    # T, KH, D, gs, page
    (1, 1, 64, 32, 16),
    (1, 8, 128, 128, 16),
    (5, 3, 96, 32, 32),
    (9, 2, 96, 96, 16),
    (33, 8, 128, 32, 64),
    (61, 8, 128, 64, 16),
    (17, 1, 256, 256, 128),
    (40, 2, 256, 64, 256),
    (1000, 5, 64, 64, 16),
]


def empty_cache(gq4, pages, KH, page, D, gs):
    """A pool filled with a pattern that no write leaves behind."""
    c = gq4.kv_cache(pages, KH, page, D, gs)
    c[0].fill_(0x5A5A5A5A)
    c[2].fill_(0x5A5A5A5A)
    c[1].fill_(-7.5)
    c[3].fill_(-7.5)
    return c


def check_cache(c, k, v, slots, page, gs):
    """Written rows equal the quantiser's, bit for bit; every other row is untouched."""
    arrays = [host(t) for t in c]
    want = [np.full(a.shape, 0x5A5A5A5A, np.uint32) if i % 2 == 0 else np.full(a.shape, -7.5, np.float32)
            for i, a in enumerate(arrays)]
    for side, x in enumerate((k, v)):
        codes, sz = R.quantise(x, gs)
        words = R.pack(codes, side == 0)
        for t, s in enumerate(slots):
            if s < 0 or s >= arrays[0].shape[0] * page:
                continue
            want[2 * side][s // page, :, s % page] = words[t]
            want[2 * side + 1][s // page, :, s % page] = sz[t]
    for got, ref in zip(arrays, want):
        got, ref = got.view(np.uint32), ref.view(np.uint32)
        nan = np.isnan(got.view(np.float32)) & np.isnan(ref.view(np.float32))
        assert np.all((got == ref) | nan)


@pytest.mark.parametrize("T,KH,D,gs,page", CACHE_CASES)
def test_append_and_gather(gq4, T, KH, D, gs, page):
    g = I.rng(2110, T, KH, D, gs, page)
    k = (g.standard_normal((T, KH, D)) * np.exp(g.standard_normal((KH, D)))).astype(np.float32)
    v = g.standard_normal((T, KH, D)).astype(np.float32)
    pages = T // page + 4
    slots = g.permutation(pages * page)[:T].astype(np.int32)
    c = empty_cache(gq4, pages, KH, page, D, gs)
    gq4.kv_append(dev(k), dev(v), dev(slots), *c, gs)
    torch.cuda.synchronize()
    check_cache(c, k, v, slots, page, gs)
    ko, vo = Guarded((T, KH, D)), Guarded((T, KH, D))
    gq4.kv_gather(dev(slots), *c, gs, k_out=ko.t, v_out=vo.t)
    torch.cuda.synchronize()
    ko.check(), vo.check()
    for got, x in ((ko.t, k), (vo.t, v)):
        codes, sz = R.quantise(x, gs)
        s, z = np.repeat(sz[..., 0], gs, -1), np.repeat(sz[..., 1], gs, -1)
        assert np.array_equal(host(got), (codes.astype(np.float32) - z) * s)
    assert gq4.device_error() == 0


@pytest.mark.parametrize("T,KH,D,gs,page", [(3000, 1, 64, 64, 16), (1025, 3, 96, 32, 32), (2, 1024, 64, 32, 16),
                                            (1500, 5, 256, 64, 64)])
def test_append_and_gather_many_rows(gq4, T, KH, D, gs, page):
    """Blocks that take several tokens, or a share of one with very many heads."""
    test_append_and_gather(gq4, T, KH, D, gs, page)


def test_append_strided_rows_skipped_and_bad_slots(gq4):
    T, KH, D, gs, page, pages = 6, 2, 64, 32, 16, 3
    g = I.rng(2111)
    x = g.standard_normal((T, 3 * KH, D)).astype(np.float32)
    fused = dev(x)
    k, v = fused[:, KH:2 * KH], fused[:, 2 * KH:]
    slots = np.array([-1, 5, pages * page, 47, -2**31, 2**31 - 1], np.int32)
    c = empty_cache(gq4, pages, KH, page, D, gs)
    gq4.kv_append(k, v, dev(slots), *c, gs)
    torch.cuda.synchronize()
    check_cache(c, x[:, KH:2 * KH], x[:, 2 * KH:], slots, page, gs)
    assert gq4.device_error(clear=True) == 1 << 6
    ko = torch.full((T, KH, D), 3.0, device="cuda")
    vo = torch.full((T, KH, D), 3.0, device="cuda")
    gq4.kv_gather(dev(slots), *c, gs, k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    assert gq4.device_error(clear=True) == 1 << 6
    for o in (host(ko), host(vo)):
        assert np.all(o[[0, 4]] == 3.0)
        assert np.isnan(o[[2, 5]]).all()
        assert np.isfinite(o[[1, 3]]).all() and np.all(o[[1, 3]] != 3.0)


def test_append_edge_groups(gq4):
    """Constant, signed-zero and tiny groups; non-finite ones become NaN rows and set bit 3."""
    KH, D, gs, page = 1, 64, 32, 16
    k = np.zeros((5, KH, D), np.float32)
    k[0] = 2.5
    k[1, 0, ::2] = -0.0
    k[2, 0, 3] = 1e-44
    k[3, 0, 5] = np.nan
    k[3, 0, 40] = 1.0
    k[4, 0, :] = np.linspace(-3e38, 3e38, D)
    v = I.rng(2112).standard_normal(k.shape).astype(np.float32)
    v[4, 0, 1] = np.inf
    slots = np.arange(5, dtype=np.int32)
    c = empty_cache(gq4, 1, KH, page, D, gs)
    gq4.device_error(clear=True)
    gq4.kv_append(dev(k), dev(v), dev(slots), *c, gs)
    torch.cuda.synchronize()
    check_cache(c, k, v, slots, page, gs)
    assert gq4.device_error(clear=True) == 1 << 3


def test_empty_calls(gq4):
    c = gq4.kv_cache(1, 2, 16, 64, 32)
    e = torch.empty((0, 2, 64), device="cuda")
    s = torch.empty(0, dtype=torch.int32, device="cuda")
    gq4.kv_append(e, e, s, *c, 32)
    k, v = gq4.kv_gather(s, *c, 32)
    assert tuple(k.shape) == (0, 2, 64)
    gq4.head_norm_rope(e, e, s, torch.ones(32, device="cuda"))
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# Book-keeping
# ---------------------------------------------------------------------------

def run_plan(gq4, past, new, table, free, count, T, page, in_place=False):
    B = len(past)
    d = [dev(np.asarray(a, np.int32)) for a in (past, new, table, free, [count])]
    outs = {"query_start": B + 1, "positions": T, "slots": T, "seq_lens": B, "free_count_out": 1}
    guards = {n: torch.full((s + 16,), -77, dtype=torch.int32, device="cuda") for n, s in outs.items()}
    views = {n: guards[n][8:8 + s] for n, s in outs.items()}
    if in_place:
        views["seq_lens"], views["free_count_out"] = d[0], d[4]
    got = gq4.kv_plan(d[0], d[1], d[2], d[3], d[4], T, page, **views)
    torch.cuda.synchronize()
    for n, s in outs.items():
        f = host(guards[n])
        assert np.all(f[:8] == -77) and np.all(f[8 + s:] == -77), n
    ref = R.plan(np.asarray(past), np.asarray(new), np.asarray(table), np.asarray(free), count, T, page)
    for a, b in zip((d[2], *got), ref[:-1]):
        assert np.array_equal(host(a), b), (host(a), b)
    assert (gq4.device_error(clear=True) == 1 << 7) == ref[-1]


def plan_inputs(B, past_most, new_most, page, width, spare, seed):
    g = I.rng(2120, B, past_most, new_most, page, seed)
    past = g.integers(0, past_most + 1, B)
    new = g.integers(0, new_most + 1, B)
    had = (past + page - 1) // page
    need = (past + new + page - 1) // page - had
    ids = g.permutation(int(had.sum() + need.sum()) + max(spare, 0) + 8).astype(np.int32)
    table = np.full((B, width), -9, np.int32)
    at = 0
    for b in range(B):
        table[b, :had[b]] = ids[at:at + had[b]]
        at += had[b]
    free = ids[at:]
    return past, new, table, free, int(need.sum()) + spare


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,past_most,new_most,page,pad", [
    (1, 0, 1, 16, 0), (1, 100, 300, 16, 7), (64, 4096, 1, 16, 0), (3, 50, 0, 32, 5), (1024, 40, 3, 16, 1),
    (1025, 300, 40, 64, 100), (5000, 64, 5, 16, 3), (7, 2000, 428, 256, 11)])
def test_plan(gq4, B, past_most, new_most, page, pad, in_place):
    width = (past_most + new_most + page - 1) // page + 1
    past, new, table, free, count = plan_inputs(B, past_most, new_most, page, width, 4, 0)
    run_plan(gq4, past, new, table, free, count, int(new.sum()) + pad, page, in_place)


def test_plan_refusals(gq4):
    """Out of pages, of rows, of table columns; negative lengths; counts beyond the list."""
    B, page = 40, 16
    past, new, table, free, count = plan_inputs(B, 90, 60, page, 11, 0, 1)
    T = int(new.sum())
    run_plan(gq4, past, new, table, free, count - 17, T, page)         # the list runs out
    run_plan(gq4, past, new, table, free, 0, T, page)
    run_plan(gq4, past, new, table, free, -5, T, page)                 # a count below 0 counts as 0
    run_plan(gq4, past, new, table, free[:9], 10**9, T, page)          # and above the list as its length
    run_plan(gq4, past, new, table, free, count, T - 100, page)        # rows past T
    run_plan(gq4, past, new, table, free, count, 0, page)
    run_plan(gq4, past, new, table[:, :6], free, count, T, page)       # the table's row is full
    p, n = past.copy(), new.copy()
    p[3], n[7], n[8] = -4, -1, 2**31 - 1
    run_plan(gq4, p, n, table, free, count, T, page)
    p[5], n[5] = 2**31 - 1, 2**31 - 1
    run_plan(gq4, p, n, table, free, count, T, page)
    run_plan(gq4, past, new, table, free, count, T, page)              # and all is well again


def test_plan_advances_its_own_state_in_a_graph(gq4):
    """A captured step with seq_lens = past_lens and free_count_out = free_count, replayed."""
    B, page, steps, width = 5, 16, 40, 8
    past, _, table, _, _ = plan_inputs(B, 20, 0, page, width, 0, 2)
    free = np.arange(100, 100 + B * width, dtype=np.int32)
    new = np.ones(B, np.int32)
    d = [dev(np.asarray(a, np.int32)) for a in (past, new, table, free, [len(free)])]
    outs = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (B + 1, B, B)]

    def step():
        gq4.kv_plan(d[0], d[1], d[2], d[3], d[4], B, page, seq_lens=d[0], query_start=outs[0], positions=outs[1],
                    slots=outs[2], free_count_out=d[4])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    count = len(free)
    for _ in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        table, past, starts, pos, slots, count, _ = R.plan(past, new, table, free, count, B, page)
        count = int(count[0])
        for a, b in zip((d[2], d[0], *outs, d[4]), (table, past, starts, pos, slots, [count])):
            assert np.array_equal(host(a), b)
    assert gq4.device_error() == 0
