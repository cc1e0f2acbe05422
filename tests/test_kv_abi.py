"""Refusals of the entry points between the QKV product and the output
projection, on the host: made-up device addresses, every call invalid, nothing
launched (as in tests/test_abi.py).  Also the layout helpers of tests/kv_ref.py
and the binding's own checks."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from tests import kv_ref as R
from tests.gpu_util import gq4_module
from tests.test_abi import ROOT, addr, no_gpu_only


@pytest.fixture(scope="module")
def gq4():
    return gq4_module()


def test_struct_layouts_match_header(gq4, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "layout.c"
    src.write_text(r"""
#include <stddef.h>
#include <stdio.h>
#include "gq4.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu %zu\n", sizeof(gq4_rope), offsetof(gq4_rope, eps), offsetof(gq4_rope, inv_freq),
         sizeof(gq4_kv_cache), offsetof(gq4_kv_cache, group_size), offsetof(gq4_kv_cache, Kq),
         offsetof(gq4_kv_cache, V_sz));
  return 0;
}
""")
    exe = tmp_path / "layout"
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), "-I", cuda_inc, str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    P, C = gq4.Rope, gq4.KVCache
    assert got == [ctypes.sizeof(P), P.eps.offset, P.inv_freq.offset, ctypes.sizeof(C), C.group_size.offset,
                   C.Kq.offset, C.V_sz.offset]


def rope(gq4, T=4, H=8, KH=2, D=64, rot=64, inter=0, eps=1e-6, pos=None, q=None, ldq=512, k=None, ldk=128, qo=None,
         ldqo=512, ko=None, ldko=128, gain=None, inv=None, no_pos=False):
    r = gq4.Rope(gain, None, eps, rot, inter, inv or addr(9))
    return gq4.lib.gq4_head_norm_rope(T, H, KH, D, ctypes.byref(r), None if no_pos else pos or addr(0), q or addr(1),
                                      ldq, k or addr(2), ldk, qo or addr(3), ldqo, ko or addr(4), ldko, None)


@no_gpu_only
def test_rope_checks(gq4):
    bad = gq4.ERR_INVALID_ARG
    for kw in (dict(T=-1), dict(H=-1), dict(H=0, KH=0), dict(H=1025, ldq=1025 * 64, ldqo=1025 * 64), dict(D=60),
               dict(D=0), dict(D=520, ldq=8192, ldk=8192, ldqo=8192, ldko=8192), dict(rot=72), dict(rot=4),
               dict(rot=-8), dict(inter=2), dict(eps=-1.0), dict(eps=float("nan")), dict(no_pos=True),
               dict(ldq=511), dict(ldq=514), dict(ldk=64), dict(ldqo=8)):
        assert rope(gq4, **kw) == bad, kw
    assert gq4.lib.gq4_head_norm_rope(1, 1, 0, 64, None, addr(0), addr(1), 64, None, 0, addr(3), 64, None, 0, None) == bad
    assert rope(gq4, q=addr(1, 4)) == gq4.ERR_MISALIGNED
    assert rope(gq4, gain=addr(5, 8)) == gq4.ERR_MISALIGNED
    assert rope(gq4, pos=addr(0, 2)) == gq4.ERR_MISALIGNED
    # q_out shifted into q, over the positions, over k_out; in place with another ld
    assert rope(gq4, qo=addr(1, 256)) == gq4.ERR_ALIAS
    assert rope(gq4, pos=addr(3, 16)) == gq4.ERR_ALIAS
    assert rope(gq4, ko=addr(3)) == gq4.ERR_ALIAS
    assert rope(gq4, q=addr(1), qo=addr(1), ldqo=516) == gq4.ERR_ALIAS
    # column blocks of one matrix that do share columns
    base = addr(1).value
    assert rope(gq4, q=addr(1), ldq=700, qo=addr(1), ldqo=700, k=ctypes.c_void_p(base + 4 * 508), ldk=700,
                ko=ctypes.c_void_p(base + 4 * 508), ldko=700) == gq4.ERR_ALIAS
    assert rope(gq4, T=0, no_pos=True) == gq4.OK


def cache(gq4, P=10, S=16, H=2, D=64, gs=32, Kq=None, K_sz=None, Vq=None, V_sz=None):
    return gq4.KVCache(P, S, H, D, gs, Kq or addr(20), K_sz or addr(21), Vq or addr(22), V_sz or addr(23))


BAD_CACHES = [dict(P=0), dict(S=8), dict(S=24), dict(S=512), dict(H=0), dict(D=48), dict(D=0), dict(gs=16),
              dict(gs=48), dict(gs=0), dict(P=1 << 28, S=16)]


@no_gpu_only
def test_append_and_gather_checks(gq4):
    lib, bad = gq4.lib, gq4.ERR_INVALID_ARG

    def append(c, T=4, k=None, ldk=128, v=None, ldv=128, slots=None):
        return lib.gq4_kv_append(T, ctypes.byref(c), k or addr(1), ldk, v or addr(2), ldv, slots or addr(3), None)

    def gather(c, T=4, slots=None, k=None, v=None):
        return lib.gq4_kv_gather(T, ctypes.byref(c), slots or addr(3), k or addr(1), v or addr(2), None)
    for kw in BAD_CACHES:
        assert append(cache(gq4, **kw)) == bad, kw
        assert gather(cache(gq4, **kw)) == bad, kw
    for D in (32, 160, 192, 512):
        assert append(cache(gq4, D=D), ldk=4096, ldv=4096) == gq4.ERR_UNSUPPORTED
    null = cache(gq4)
    null.Vq = None
    assert append(null) == bad and gather(null) == bad
    assert append(cache(gq4, K_sz=addr(21, 8))) == gq4.ERR_MISALIGNED
    c = cache(gq4)
    assert append(c, T=-1) == bad and append(c, ldk=127) == bad and append(c, ldv=64) == bad
    assert append(c, k=addr(1, 4)) == gq4.ERR_MISALIGNED
    assert append(c, slots=addr(3, 2)) == gq4.ERR_MISALIGNED
    assert append(c, k=addr(20, 64)) == gq4.ERR_ALIAS        # rows inside the pool
    assert append(c, slots=addr(23)) == gq4.ERR_ALIAS
    assert append(cache(gq4, Vq=addr(20, 256))) == gq4.ERR_ALIAS
    assert gather(c, k=addr(2)) == gq4.ERR_ALIAS             # k_out over v_out
    assert gather(c, v=addr(22, 16)) == gq4.ERR_ALIAS
    assert gather(c, k=addr(1, 8)) == gq4.ERR_MISALIGNED
    assert append(c, T=0) == gq4.OK and gather(c, T=0) == gq4.OK


@no_gpu_only
def test_plan_checks(gq4):
    def plan(B=4, T=8, page=16, width=5, n_free=6, **at):
        names = ["past", "new", "table", "free", "count", "count_out", "lens", "starts", "positions", "slots"]
        p = [at.get(n, addr(i)) for i, n in enumerate(names)]
        return gq4.lib.gq4_kv_plan(B, T, page, width, n_free, *p, None)
    bad = gq4.ERR_INVALID_ARG
    for kw in (dict(B=0), dict(B=65537), dict(T=-1), dict(page=8), dict(page=48), dict(width=0), dict(n_free=-1),
               dict(width=1 << 28), dict(past=None), dict(table=None), dict(free=None), dict(count=None),
               dict(count_out=None), dict(lens=None), dict(starts=None), dict(slots=None)):
        assert plan(**kw) == bad, kw
    assert plan(table=addr(2, 2)) == gq4.ERR_MISALIGNED
    assert plan(lens=addr(1)) == gq4.ERR_ALIAS               # lens over new_lens
    assert plan(lens=addr(0, 4)) == gq4.ERR_ALIAS            # partly over past_lens
    assert plan(positions=addr(9, 4)) == gq4.ERR_ALIAS
    assert plan(count_out=addr(3, 8)) == gq4.ERR_ALIAS
    assert plan(table=addr(3, -16)) == gq4.ERR_ALIAS


@no_gpu_only
def test_attention_checks(gq4):
    lib, bad = gq4.lib, gq4.ERR_INVALID_ARG
    need = gq4.kv_attention_workspace_bytes(4, 8, 2, 64)
    assert need > 0

    def attn(c=None, B=2, T=4, H=8, width=3, mq=2, ml=0, q=None, ldq=512, starts=None, lens=None, table=None,
             scale=0.1, window=0, out=None, ldo=512, ws=None, wb=None):
        c = c or cache(gq4)
        return lib.gq4_kv_attention(B, T, H, width, mq, ml, ctypes.byref(c), q or addr(1), ldq, starts or addr(2),
                                    lens or addr(3), table or addr(4), scale, window, out or addr(5), ldo,
                                    ws or addr(6), need if wb is None else wb, None)
    for kw in BAD_CACHES:
        assert attn(cache(gq4, **kw)) == bad, kw
    assert attn(cache(gq4, D=192), ldq=4096, ldo=4096) == gq4.ERR_UNSUPPORTED
    for kw in (dict(B=0), dict(B=65537), dict(T=-1), dict(H=0), dict(H=7), dict(H=1026, ldq=1026 * 64), dict(width=0),
               dict(width=1 << 28), dict(mq=-1), dict(ml=-1), dict(window=-1), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(ldq=510), dict(ldo=256), dict(wb=need - 1)):
        assert attn(**kw) == bad, kw
    assert attn(q=addr(1, 8)) == gq4.ERR_MISALIGNED
    assert attn(lens=addr(3, 1)) == gq4.ERR_MISALIGNED
    assert attn(ws=addr(6, 128)) == gq4.ERR_MISALIGNED
    assert attn(out=addr(1)) == gq4.ERR_ALIAS
    assert attn(out=addr(20, 32)) == gq4.ERR_ALIAS
    assert attn(ws=addr(5, 256)) == gq4.ERR_ALIAS
    assert attn(T=0) == gq4.OK and attn(mq=0) == gq4.OK


def test_binding_refuses(gq4):
    x = torch.zeros(2, 2, 64)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gq4.head_norm_rope(x, None, i, None)
    with pytest.raises(ValueError, match="q or k"):
        gq4.head_norm_rope(None, None, i, None)
    c = (torch.zeros(1, 2, 16, 8, dtype=torch.int32), torch.zeros(1, 2, 16, 2, 2)) * 2
    for call in (lambda: gq4.kv_append(x, x, i, *c, 32), lambda: gq4.kv_gather(i, *c, 32),
                 lambda: gq4.kv_attention(x, i, i, i, *c, 32, scale=1.0, max_query=1),
                 lambda: gq4.kv_plan(i, i, i, i, i, 2, 16)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="group_size"):
        gq4.kv_cache(1, 1, 16, 64, 48, device="cpu")


@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_layout_restatement(D):
    """The restated layout is a permutation of a row's nibbles, and packing inverts."""
    for keys in (True, False):
        word, bit = R.places(D, keys)
        assert sorted(8 * word + bit // 4) == list(range(D))
        codes = np.random.default_rng(5).integers(0, 16, (3, D), dtype=np.uint8)
        assert np.array_equal(R.unpack(R.pack(codes, keys), keys), codes)


def test_plan_restatement():
    """A worked step: pages of 16; request 0 fills its page, request 1 starts, request 2 idles."""
    table = np.array([[7, -1], [-1, -1], [3, -1]], np.int32)
    out = R.plan([15, 0, 4], [2, 17, 0], table, np.array([9, 8, 6, 5]), 4, 20, 16)
    t, lens, starts, pos, slots, count, refused = out
    assert t.tolist() == [[7, 5], [6, 8], [3, -1]] and lens.tolist() == [17, 17, 4]
    assert starts.tolist() == [0, 2, 19, 19] and count.tolist() == [1] and not refused
    assert pos.tolist() == [15, 16] + list(range(17)) + [0]
    assert slots.tolist() == [127, 80] + list(range(96, 112)) + [128, -1]
