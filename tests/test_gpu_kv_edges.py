"""GPU tests of the cache calls' edges: page ids that are none, refusals that
write nothing, the largest step, outputs allocated for another stream."""

import numpy as np
import pytest
import torch

from tests.gpu_util import dev, gq4_module, host, requires_cuda
from tests.test_gpu_attention import FILL, Setup

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def gq4():
    g = gq4_module()
    g.device_error(clear=True)
    return g


def plan(gq4, past, new, table, free, count, T, page, **kw):
    d = [dev(np.asarray(a, np.int32)) for a in (past, new, table, free, [count])]
    got = gq4.kv_plan(*d, T, page, **kw)
    torch.cuda.synchronize()
    return [host(t) for t in (d[2], *got)]


@pytest.mark.parametrize("page", [16, 256])
def test_page_ids_that_name_no_slot(gq4, page):
    """An id below 0, or whose slots pass 2^31, on the free list or in the table: the token's slot is
    2^31 - 1, outside any pool, which the writer reports; the largest id that has slots is used."""
    top = 2**31 // page
    free = [top - 1, top, 2**32 // page - 2**31 // page, -1, -2**31, 5, 2**31 - 1]
    new = [1] * len(free)
    # granted off the end of the list
    table, lens, starts, pos, slots, left = plan(gq4, [0] * 7, new, np.full((7, 1), -9), free, 7, 7, page)
    want = [2**31 - 1 if not 0 <= i < top else i * page for i in free[::-1]]
    assert slots.tolist() == want and table[:, 0].tolist() == free[::-1] and left[0] == 0
    # already in the table
    table, lens, starts, pos, slots, left = plan(gq4, [3] * 7, new, np.array(free)[:, None], [1], 1, 7, page)
    assert slots.tolist() == [2**31 - 1 if not 0 <= i < top else i * page + 3 for i in free]
    assert gq4.device_error(clear=True) == 0
    c = gq4.kv_cache(1, 1, page, 64, 32)
    x = torch.ones((1, 1, 64), device="cuda")
    gq4.kv_append(x, x, dev(np.array([2**31 - 1], np.int32)), *c, 32)
    torch.cuda.synchronize()
    assert gq4.device_error(clear=True) == 1 << 6
    assert all(not bool(t.any()) for t in c)


def test_a_request_too_long_is_refused_without_new_tokens_too(gq4):
    """past + new beyond the table's row sets bit 7, whether or not the request has new tokens."""
    table, lens, starts, pos, slots, left = plan(gq4, [33, 5], [0, 1], [[1, 2], [3, -9]], [7], 1, 1, 16)
    assert gq4.device_error(clear=True) == 1 << 7
    assert lens.tolist() == [33, 6] and starts.tolist() == [0, 0, 1] and slots.tolist() == [3 * 16 + 5]
    # at its end without new ones, or behind rows that were cut: nothing is refused there
    plan(gq4, [32, 5], [0, 0], [[1, 2], [3, -9]], [7], 1, 0, 16)
    assert gq4.device_error(clear=True) == 0


def test_the_largest_step(gq4):
    """2^31 - 1 token rows (17 GB of positions and slots), nearly all of them of no request."""
    T = 2**31 - 1
    out = [torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2)]
    for o in out:
        o.fill_(-77)
    got = gq4.kv_plan(*[dev(np.asarray(a, np.int32)) for a in ([7], [3], [[4]], [1], [1])], T, 16, positions=out[0],
                      slots=out[1])
    torch.cuda.synchronize()
    assert host(got[1]).tolist() == [0, 3]
    assert host(out[0][:3]).tolist() == [7, 8, 9] and host(out[1][:3]).tolist() == [71, 72, 73]
    for o, rest in zip(out, (0, -1)):
        for part in o[3:].split(2**28):
            assert int(part.min()) == rest and int(part.max()) == rest
    assert gq4.device_error(clear=True) == 0


def test_outputs_allocated_for_another_stream(gq4):
    """What a call allocates may be memory whose last use is still under way on the current stream:
    the call's own stream waits for it, and it is not handed out again while that stream uses it."""
    s = Setup([1, 1], [3000, 900], 8, 2, 128, 128, 16)
    clean = s.run(gq4)
    live = int(s.starts[-1])
    args, q = s.dev(), dev(s.q)
    k = torch.ones((64, 2, 128), device="cuda")
    slots = torch.arange(64, dtype=torch.int32, device="cuda")
    cache = gq4.kv_cache(4, 2, 16, 128, 128)
    gq4.kv_append(k, k, slots, *cache, 128)
    inv = torch.ones(64, device="cuda")
    lens, new = (torch.full((1,), n, dtype=torch.int32, device="cuda") for n in (0, 64))
    table = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    free, count = torch.arange(4, dtype=torch.int32, device="cuda"), torch.full((1,), 4, dtype=torch.int32,
                                                                                device="cuda")
    side = torch.cuda.Stream()
    calls = {
        "attention": lambda: (gq4.kv_attention(q, *args, scale=s.scale, max_query=1, max_len=3000, stream=side),),
        "rope": lambda: gq4.head_norm_rope(k, None, slots, inv, stream=side)[:1],
        "gather": lambda: gq4.kv_gather(slots, *cache, 128, stream=side),
        "plan": lambda: gq4.kv_plan(lens, new, table, free, count, 64, 16, stream=side),
    }
    for name, call in calls.items():
        torch.cuda.synchronize()
        want = [host(t) for t in call()]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        # blocks of every size the call may ask for, freed with a write of theirs under way
        held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
                (512, 1024, 2048, 4096, 20480, 65536, gq4.kv_attention_workspace_bytes(s.T, 8, 2, 128)) for _ in "ab"]
        torch.cuda._sleep(100_000_000)
        for t in held:
            t.fill_(255)
        del held, t
        got = call()
        side.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            a = host(a)
            if name == "attention":
                a, b = a[:live], clean[:live]
            assert np.array_equal(a, b), name
