"""GPU tests of steps in which kv_plan refuses requests: trees and accepted paths by the planned slots, and a speculative
loop whose pool runs dry."""

import numpy as np
import pytest
import torch

from int4_group_quantized_quant_gb300 import inputs as I
from tests import kv_ref as R
from tests import mask_ref as M
from tests.gpu_util import dev, gq4_module, host, requires_cuda
from tests.test_gpu_trees import Accept, check_rows, inv_freq

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def gq4():
    g = gq4_module()
    g.device_error(clear=True)
    return g


def ints(*a):
    return dev(np.array(a, np.int32))


@pytest.mark.parametrize("counts,path", [([0, 2], [[0, 0, 0], [0, 1, 0]]), ([3, 2], [[0, 2, 4], [1, 3, 0]]),
                                         ([-1, 1], [[9, 9, 9], [7, 0, 0]]), ([8, 3], None), ([0, 0], None)])
def test_refused_request_stays(gq4, counts, path):
    """32 tokens that fill two pages and an empty list: 8 more are refused, and none of the 32 is lost, whatever its count
    and path say.  Its neighbour has room and loses what is not accepted."""
    KH, D, gs, page, n = 2, 64, 32, 16, 8
    g = I.rng(2700)
    cache = gq4.kv_cache(4, KH, page, D, gs)
    k = dev(g.standard_normal((64, KH, D)).astype(np.float32))
    gq4.kv_append(k, k, dev(np.arange(64, dtype=np.int32)), *cache, gs)
    before = [host(t).copy() for t in cache]
    table, free = ints([1, 3, -1], [2, -1, -1]), ints(-7, -7)
    lens, count = ints(32, 5), ints(0)
    _, starts, _, slots, _ = gq4.kv_plan(lens, ints(n, n), table, free, count, 2 * n, page, seq_lens=lens, free_count_out=count)
    assert gq4.device_error(clear=True) == 1 << 7
    assert host(lens).tolist() == [32, 13] and host(slots).tolist() == [-1] * n + list(range(37, 45))
    up = np.array([-1, 0, 0, 1, 1, 2, 2, 3], np.int32)
    # (parents of a request that has no nodes may be anything)
    pos, tree = gq4.kv_tree(dev(np.concatenate([up + 9, up])), starts, lens, 1, slots=slots)
    want_pos, want, _ = M.tree(up, [0, n], [13], 1)
    assert host(pos).tolist() == [0] * n + want_pos.tolist()
    assert np.array_equal(host(tree).view(np.uint32), np.concatenate([np.zeros((n, 1), np.uint32), want]))
    gq4.kv_accept(None if path is None else dev(np.array(path, np.int32)), ints(*counts), starts, lens, table, free, count,
                  *cache, gs, seq_lens_out=lens, free_count_out=count, slots=slots)
    moved = dict(enumerate(path[1][:counts[1]])) if path is not None else {}
    refused = any(not j < x < n for x, j in zip(moved.values(), [-1] + list(moved.values())))
    assert gq4.device_error(clear=True) == (1 << 11 if refused else 0)
    assert host(lens).tolist() == [32, 13 if refused else 5 + counts[1]] and host(count).tolist() == [0]
    assert host(free).tolist() == [-7, -7]
    for a, t in zip(before, cache):
        want = a.copy()
        for to, at in moved.items():
            if not refused:
                want[2, :, 5 + to] = a[2, :, 5 + at]
        assert np.array_equal(host(t), want)


def test_rows_out_of_the_slots(gq4):
    """Rows that are not within the slots given: the request is refused, bit 11; without rows nothing is looked at."""
    KH, D, gs, page = 1, 64, 32, 16
    cache = gq4.kv_cache(4, KH, page, D, gs)
    table, free, count = ints([0, 1], [2, 3]), ints(-7, -7, -7), ints(0)
    for starts, slots, lens, refused in (([0, 3, 6], [5, 6, 7, 40, 41], [9, 9], [False, True]),
                                         ([-1, 2, 5], [5, 6, 7, 40, 41], [9, 9], [True, False]),
                                         ([0, 0, 0], [], [9, 9], [False, False]), ([0, 1, 1], [], [9, 9], [True, False])):
        out, left = gq4.kv_accept(None, ints(0, 0), ints(*starts), ints(*lens), table, free, count, *cache, gs,
                                  slots=ints(*slots))
        n = np.diff(starts)
        assert host(out).tolist() == [x if bad else x - int(m) for x, m, bad in zip(lens, n, refused)]
        assert gq4.device_error(clear=True) == (1 << 11 if any(refused) else 0) and host(left).tolist() == [0]


@pytest.mark.parametrize("sizes,kw", [([int(n) for n in np.arange(2500) % 9], dict(KH=1)),
                                      ([33, 7, 0, 60, 12, 5], dict(KH=8, D=128, gs=64)), ([256, 3, 250, 17], dict(KH=2))])
@pytest.mark.parametrize("line", [False, True])
def test_many_requests_some_refused(gq4, sizes, kw, line):
    """Every third request without slots, of any count and path: it stays, the others are as without it."""
    a = Accept(sizes, **kw)
    B, starts = len(sizes), a.starts
    lost = np.arange(B) % 3 == 1
    slots = np.arange(100, 100 + starts[-1], dtype=np.int32)
    for b in np.nonzero(lost)[0]:
        slots[starts[b]:starts[b + 1]] = -1
    # the rule on the others alone: a lost request has no rows there, and nothing is accepted of it
    sizes_left = np.where(lost & (np.array(sizes) > 0), 0, sizes)
    counts = np.where(sizes_left > 0, a.counts, 0)
    path = None if line else a.path
    lens, free, count, moves, refused = M.accept(path, counts, np.concatenate([[0], np.cumsum(sizes_left)]), a.lens, a.table,
                                                 a.free, a.count_free, a.pages, a.page)
    assert not refused
    arrays, old = [x.copy() for x in a.cache.arrays()], a.cache.arrays()
    for b, src, dst in moves:
        (ps, s), (pd, d) = ((a.table[b, t // a.page], t % a.page) for t in (src, dst))
        for x, o in zip(arrays, old):
            x[pd, :, d] = o[ps, :, s]
    given = np.where(lost & (np.array(sizes) > 0), np.arange(B) % 7 - 2, a.counts).astype(np.int32)
    cache, free_dev = [dev(x) for x in a.cache.arrays()], dev(a.free)
    got = gq4.kv_accept(None if line else dev(path), dev(given), dev(starts), dev(a.lens), dev(a.table), free_dev,
                        ints(a.count_free), *cache, a.gs, slots=dev(slots))
    torch.cuda.synchronize()
    assert gq4.device_error(clear=True) == 0
    assert np.array_equal(host(got[0]), lens) and host(got[1]).tolist() == [count] and np.array_equal(host(free_dev), free)
    for x, c in zip(arrays, cache):
        assert np.array_equal(host(c).view(np.uint32), x.view(np.uint32))
    # and the bits of the same trees
    parents = np.concatenate([M.random_parents(I.rng(5, b), n) for b, n in enumerate(sizes)]).astype(np.int32)
    want_pos, want, refused = M.tree(parents, starts, a.lens, 8, 5, 9)
    assert not refused
    pos, tree = gq4.kv_tree(dev(parents), dev(starts), dev(a.lens), 8, window=5, sinks=9, slots=dev(slots))
    want_pos[slots < 0], want[slots < 0] = 0, 0
    assert np.array_equal(host(pos), want_pos) and np.array_equal(host(tree).view(np.uint32), want)
    assert gq4.device_error() == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 4)])
@pytest.mark.parametrize("line", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_loop_whose_pool_runs_dry(gq4, window, sinks, line, graph):
    """Steps of drafted trees (or lines) of which some are refused for want of pages or of room in the table; requests end
    and give their pages back.  Every committed token reads back as written, attention is that of the rows in the cache,
    no page is lost or held twice, and only kv_plan reports anything."""
    H, KH, D, gs, page, B, n, words, pages, width, steps = 4, 2, 64, 32, 16, 4, 11, 1, 8, 3, 24
    g = I.rng(2710, window, line)
    inv, gain = inv_freq(D), g.uniform(0.5, 1.5, D).astype(np.float32)
    cache = gq4.kv_cache(pages, KH, page, D, gs)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count = dev(np.arange(pages, dtype=np.int32)), ints(pages)
    lens, dinv, dgain = ints(*[0] * B), dev(inv), dev(gain)
    tokens = [[] for _ in range(B)]             # (k, v) of what stays
    T = B * n
    xin, parents = torch.zeros((T, H + 2 * KH, D), device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    new, counts = ints(*[0] * B), ints(*[0] * B)
    path = torch.zeros((B, n), dtype=torch.int32, device="cuda")
    ws = torch.empty(gq4.kv_attention_workspace_bytes(T, H, KH, D, tree=True), dtype=torch.uint8, device="cuda")
    kept = {}

    def draft():
        _, st, _, slots, _ = gq4.kv_plan(lens, new, table, free, count, T, page, seq_lens=lens, free_count_out=count)
        p, tree = gq4.kv_tree(parents, st, lens, words, window=window, sinks=sinks, slots=slots)
        qr = gq4.kv_rope_append(xin[:, :H], xin[:, H:H + KH], xin[:, H + KH:], p, dinv, slots, *cache, gs, k_gain=dgain)
        out = gq4.kv_attention(qr, st, lens, table, *cache, gs, scale=D ** -0.5, max_query=n, window=window, sinks=sinks,
                               tree=tree, positions=p, workspace=ws)
        kept.update(starts=st, positions=p, slots=slots, q=qr, out=out, tree=tree)

    def accept():
        gq4.kv_accept(None if line else path, counts, kept["starts"], lens, table, free, count, *cache, gs, seq_lens_out=lens,
                      free_count_out=count, slots=kept["slots"])

    def read_back(b, tb):
        t = np.arange(len(tokens[b]))
        if len(t):
            check_rows(gq4, None, np.stack([k for k, _ in tokens[b]]), np.stack([v for _, v in tokens[b]]), t.astype(np.int32),
                       inv, tb[b, t // page] * page + t % page, cache, gs, page, None, gain, False, None)

    graphs = None
    if graph:
        side, graphs = torch.cuda.Stream(), [torch.cuda.CUDAGraph() for _ in range(2)]
        torch.cuda.synchronize()
        for gr, f in zip(graphs, (draft, accept)):
            with torch.cuda.stream(side):
                with torch.cuda.graph(gr, stream=side):
                    f()
    dry = full = 0
    for step in range(steps):
        x = g.standard_normal((T, H + 2 * KH, D)).astype(np.float32)
        news = g.integers(1, n + 1, B).astype(np.int32)
        if step % 3 == 1:
            news[int(g.integers(B))] = 0
        st = np.concatenate([[0], np.cumsum(news)])
        up = np.full(T, 77, np.int32)
        for b in range(B):
            up[st[b]:st[b + 1]] = np.arange(news[b]) - 1 if line else M.random_parents(g, int(news[b]), 4)
        for t, a in ((xin, x), (parents, up), (new, news)):
            t.copy_(dev(a))
        old = [len(t) for t in tokens]
        _, want_lens, want_st, _, want_slots, _, _ = R.plan(old, news, host(table), host(free), host(count)[0], T, page)
        graphs[0].replay() if graph else draft()
        torch.cuda.synchronize()
        lost = (want_lens == old) & (news > 0)
        dry += int((lost & (np.array(old) + news <= width * page)).sum())
        full += int((np.array(old) + news > width * page).sum())
        assert gq4.device_error(clear=True) == (1 << 7 if lost.any() else 0)
        now, tb, pos = host(lens), host(table), host(kept["positions"])
        assert np.array_equal(now, want_lens) and np.array_equal(host(kept["starts"]), want_st)
        assert np.array_equal(host(kept["slots"]), want_slots)
        bits = host(kept["tree"]).view(np.uint32)
        for b in range(B):
            rows, m, L = slice(int(st[b]), int(st[b + 1])), int(news[b]), int(now[b])
            if lost[b]:
                assert np.all(pos[rows] == 0) and np.all(bits[rows] == 0)
            elif m > 0:
                want_pos, want, _ = M.tree(up[rows], [0, m], [L], words, window, sinks)
                assert np.array_equal(pos[rows], want_pos) and np.array_equal(bits[rows], want)
                t = np.arange(L)
                ks, vs = (host(a).astype(np.float64) for a in
                          gq4.kv_gather(dev((tb[b, t // page] * page + t % page).astype(np.int32)), *cache, gs))
                seen = M.sight(m, L, window, sinks, want, want_pos)
                qh, out = host(kept["q"])[rows].astype(np.float64), host(kept["out"])[rows]
                for h in range(H):
                    w = D ** -0.5 * qh[:, h] @ ks[:, h // (H // KH)].T
                    w = np.where(seen, np.exp(w - np.where(seen, w, -np.inf).max(-1, keepdims=True)), 0)
                    assert np.allclose(out[:, h], w @ vs[:, h // (H // KH)] / w.sum(-1, keepdims=True), rtol=1e-4, atol=1e-4)
        # a path from a root, from parent to child; of a refused request anything
        chosen, taken = np.zeros((B, n), np.int32), np.zeros(B, np.int32)
        for b in range(B):
            if lost[b]:
                taken[b] = (0, 3, n, -2)[step % 4]
                chosen[b] = g.integers(-2, n + 2, n)
                continue
            own, nodes = up[st[b]:st[b + 1]], []
            for _ in range(int(g.integers(2, 8))):
                below = [i for i in range(len(own)) if own[i] == (nodes[-1] if nodes else -1)]
                if not below:
                    break
                nodes.append(int(g.choice(below)))
            chosen[b, :len(nodes)], taken[b] = nodes, len(nodes)
            tokens[b] += [(x[st[b] + i, H:H + KH], x[st[b] + i, H + KH:]) for i in nodes]
        path.copy_(dev(chosen))
        counts.copy_(dev(taken))
        graphs[1].replay() if graph else accept()
        torch.cuda.synchronize()
        assert gq4.device_error(clear=True) == 0
        now, tb = host(lens), host(table)
        assert now.tolist() == [len(t) for t in tokens]
        held = [tb[b, :(now[b] + page - 1) // page].tolist() for b in range(B)]
        left = host(free)[:int(host(count)[0])].tolist()
        assert sorted(sum(held, []) + left) == list(range(pages))
        if step % 6 == 5:                       # the longest request ends
            b = int(np.argmax(now))
            read_back(b, tb)
            c = int(host(count)[0])
            free[c:c + len(held[b])] = ints(*held[b])
            count += len(held[b])
            lens[b], tokens[b] = 0, []
    assert dry >= 4 and (full >= 1 or not line)
    for b in range(B):
        read_back(b, tb)
