"""Row tiles of a tree call whose CTA gave up a wait: the last kernel leaves no row that other calls' sums went into.  That
kernel alone is run, over the workspace of a call that went well, in which CTAs are then marked as having given up; nothing
waits."""

import ctypes
import subprocess

import numpy as np
import pytest
import torch

from int4_group_quantized_quant_gb300 import build
from int4_group_quantized_quant_gb300 import inputs as I
from tests import kv_ref as R
from tests import mask_ref as M
from tests.gpu_util import dev, gq4_module, host, requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = tmp_path_factory.mktemp("undone") / "undone.so"
    subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-shared", "-o", str(so),
                    str(build.ROOT) + "/tests/undone.cu"], check=True)
    lib = ctypes.CDLL(str(so))
    lib.sums_bytes.restype = ctypes.c_longlong
    i, p = ctypes.c_int, ctypes.c_void_p
    lib.run_join.argtypes = [i] * 6 + [p, p, i, p, p, p, ctypes.c_float, p, i, p, i, i, p, ctypes.c_longlong, i, p, p, p]
    return lib


def test_rows_of_a_cta_that_gave_up(lib):
    gq4 = gq4_module()
    sizes, heads, kv_heads, D, page, words, least = [40] * 9 + [3, 100, 0, 64], 32, 8, 128, 16, 4, 64
    g, per = I.rng(2800), heads // kv_heads
    B, starts = len(sizes), np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    T = int(starts[-1]) + 2
    lens = (np.array(sizes) + g.integers(1500, 3000, B)).astype(np.int32)
    width = int(lens.max() + page - 1) // page
    pool = R.Cache(g, B * width, kv_heads, page, D, D)
    table = dev(g.permutation(B * width).reshape(B, width).astype(np.int32))
    _, bits, _ = M.tree(np.concatenate([M.random_parents(g, n) for n in sizes] + [np.zeros(2, int)]), starts, lens, words)
    arrays = [dev(a) for a in pool.arrays()]
    q, at_starts, at_lens, tree = dev(g.standard_normal((T, heads, D)).astype(np.float32)), dev(starts), dev(lens), dev(bits)
    out = torch.full((T, heads, D), 5.0, device="cuda")
    ws = torch.empty(gq4.kv_attention_workspace_bytes(T, heads, kv_heads, D, tree=True), dtype=torch.uint8, device="cuda")
    gq4.kv_attention(q, at_starts, at_lens, table, *arrays, D, scale=0.1, max_query=100, max_len=3100, out=out, workspace=ws,
                     tree=tree)
    torch.cuda.synchronize()
    clean = host(out).copy()
    ctas = min(torch.cuda.get_device_properties(0).multi_processor_count, 152)
    n_units = ((T * per + 127) // 128 + min(B, T * per // 48)) * kv_heads
    apart = lib.sums_bytes()
    cut_at = apart + (n_units + 2 * ctas) * 32
    cut = ws[cut_at:cut_at + 16 * ctas].view(torch.int32).view(ctas, 4)
    pieces_at = cut_at + 16 * ctas
    pieces = ws[pieces_at:pieces_at + ctas * 2 * 128 * (D + 2) * 4].view(torch.float32).view(ctas, 2, -1)
    cache, C = gq4.KVCache(B * width, page, kv_heads, D, D, *[t.data_ptr() for t in arrays]), ctypes.c_void_p

    def join():
        out.fill_(5.0)
        err = lib.run_join(B, T, heads, width, 100, 3100, ctypes.byref(cache), q.data_ptr(), heads * D, at_starts.data_ptr(),
                           at_lens.data_ptr(), table.data_ptr(), 0.1, tree.data_ptr(), words, out.data_ptr(), heads * D, least,
                           C(ws.data_ptr() + apart), n_units, ctas, C(cut.data_ptr()), C(pieces.data_ptr()),
                           C(torch.cuda.current_stream().cuda_stream))
        assert err == 0
        torch.cuda.synchronize()
        return host(out)

    # the workspace is read where the call keeps it: cut row tiles are joined as the call joined them
    own = host(cut)
    was = own[:, 3] >= 0
    assert was.sum() > 50 and np.all(own[was, 0] < B) and np.all(own[was, 2] < kv_heads) and np.all(own[was, 3] < ctas)
    got = join()
    joined = np.zeros((T, heads), bool)
    def rows_of(b, tile, h):
        rho = np.arange(128 * tile, min(128 * tile + 128, sizes[b] * per))
        return starts[b] + rho // per, h * per + rho % per

    for u in own[was]:
        joined[rows_of(*u[:3])] = True
    assert np.array_equal(got[joined], clean[joined]) and np.all(got[~joined] == 5.0)
    # CTAs that gave up: what their sums hold is another call's, and row tiles of theirs are not written at all
    many = np.zeros(T, bool)
    for b, n in enumerate(sizes):
        many[starts[b]:starts[b + 1]] = n * per >= least
    keep = cut.clone(), pieces.clone()
    for gone in ([0], [ctas - 1], [7, 8, 60], list(range(ctas))):
        cut.copy_(keep[0])
        pieces.copy_(keep[1])
        cut[gone, 3] = -2
        pieces[gone] = 1000.0
        got = join()
        want = np.where(many[:, None, None], np.float32(np.nan), np.float32(5.0)) + np.zeros_like(clean)
        for c in np.nonzero(was)[0]:
            if not set(gone) & set(range(c, own[c, 3] + 1)):
                want[rows_of(*own[c, :3])] = clean[rows_of(*own[c, :3])]
        assert np.array_equal(got, want, equal_nan=True), gone
        assert np.isfinite(want[many]).any() == (len(gone) < ctas)
    assert gq4.device_error(clear=True) == 0
