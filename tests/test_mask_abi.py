"""Refusals of the attention with masks on the host (made-up device addresses, every call invalid, nothing launched), the
struct's layout, and worked examples of the restatements."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from tests import mask_ref as M
from tests.gpu_util import gq4_module
from tests.test_abi import ROOT, addr, no_gpu_only
from tests.test_kv_abi import BAD_CACHES, cache


@pytest.fixture(scope="module")
def gq4():
    return gq4_module()


def test_struct_layout_matches_header(gq4, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "layout.c"
    src.write_text(r"""
#include <stddef.h>
#include <stdio.h>
#include "gq4.h"
int main(void) {
  printf("%zu %zu %zu %zu %d\n", sizeof(gq4_kv_mask), offsetof(gq4_kv_mask, tree), offsetof(gq4_kv_mask, tree_words),
         offsetof(gq4_kv_mask, positions), GQ4_MAX_TREE_WORDS);
  return 0;
}
""")
    exe = tmp_path / "layout"
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), "-I", cuda_inc, str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    K = gq4.KVMask
    assert got == [ctypes.sizeof(K), K.tree.offset, K.tree_words.offset, K.positions.offset, 8]


@no_gpu_only
def test_attention_checks(gq4):
    lib, bad = gq4.lib, gq4.ERR_INVALID_ARG
    need = gq4.kv_attention_workspace_bytes(4, 8, 2, 64, tree=True)
    c = cache(gq4)

    def attn(B=2, T=4, mq=2, q=None, table=None, scale=0.1, out=None, ws=None, wb=need, window=0, sinks=0, tree=addr(7),
             words=1, pos=addr(8), mask=True):
        m = gq4.KVMask(window, sinks, tree, words, pos)
        return lib.gq4_kv_attention_masked(B, T, 8, 3, mq, 0, ctypes.byref(c), q or addr(1), 512, addr(2), addr(3),
                                           table or addr(4), scale, ctypes.byref(m) if mask else None, out or addr(5), 512,
                                           ws or addr(6), wb, None)
    for kw in (dict(B=0), dict(T=-1), dict(mq=-1), dict(scale=float("nan")), dict(wb=need - 1), dict(window=-1),
               dict(sinks=-1), dict(sinks=-1, tree=None), dict(words=0), dict(words=9), dict(words=-1),
               dict(window=3, pos=None), dict(mask=False), dict(words=0, T=0)):
        assert attn(**kw) == bad, kw
    assert attn(tree=addr(7, 2)) == gq4.ERR_MISALIGNED
    assert attn(window=3, pos=addr(8, 1)) == gq4.ERR_MISALIGNED
    assert attn(q=addr(1, 8)) == gq4.ERR_MISALIGNED
    assert attn(tree=addr(5, 64)) == gq4.ERR_ALIAS                # bits inside the output
    assert attn(tree=addr(6, 128)) == gq4.ERR_ALIAS               # and inside the workspace
    assert attn(window=3, pos=addr(5)) == gq4.ERR_ALIAS
    assert attn(out=addr(1)) == gq4.ERR_ALIAS
    assert attn(T=0) == gq4.OK and attn(mq=0) == gq4.OK


def test_worked_tree():
    """past 4:  0 - 1 - 3, 0 - 2, and a second root 4 - 5."""
    parents = np.array([-1, 0, 0, 1, -1, 4], np.int32)
    pos, bits, refused = M.tree(parents, [0, 6], [10], 1)
    assert pos.tolist() == [4, 5, 5, 6, 4, 5] and not refused
    assert bits[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b110000]
    # a window of 2 leaves a node its parent; the first five positions stay in sight
    assert M.tree(parents, [0, 6], [10], 1, window=2)[1][:, 0].tolist() == [1, 3, 5, 0b1010, 0b10000, 0b110000]
    assert M.tree(parents, [0, 6], [10], 1, window=2, sinks=5)[1][:, 0].tolist() == bits[:, 0].tolist()
    seen = M.sight(6, 10, 3, 1, bits, pos)
    assert seen[3].tolist() == [True, False, False, False, True, True, False, True, False, False]
    assert M.sight(2, 6, 2, 1).tolist() == [[1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert M.tree(np.array([-1, 1], np.int32), [0, 2], [2], 1)[2]


@no_gpu_only
def test_rope_append_checks(gq4):
    lib, bad = gq4.lib, gq4.ERR_INVALID_ARG

    def call(c=None, T=4, H=8, rot=64, inter=0, eps=1e-6, qg=None, kg=None, pos=addr(0), inv=addr(9), q=addr(1), ldq=512,
             qo=addr(2), ldqo=512, k=addr(3), ldk=128, v=addr(4), ldv=128, slots=addr(5)):
        r = gq4.Rope(qg, kg, eps, rot, inter, inv)
        return lib.gq4_kv_rope_append(T, H, ctypes.byref(c or cache(gq4)), ctypes.byref(r), pos, q, ldq, qo, ldqo, k, ldk, v,
                                      ldv, slots, None)
    for kw in BAD_CACHES:
        assert call(cache(gq4, **kw)) == bad, kw
    assert call(cache(gq4, D=192), ldq=4096, ldqo=4096, ldk=4096, ldv=4096) == gq4.ERR_UNSUPPORTED
    for kw in (dict(T=-1), dict(H=-1), dict(H=1025, ldq=1 << 17, ldqo=1 << 17), dict(rot=4), dict(rot=72), dict(rot=-8),
               dict(inter=2), dict(eps=-1.0), dict(eps=float("nan")), dict(pos=None), dict(inv=None), dict(q=None),
               dict(qo=None), dict(k=None), dict(v=None), dict(slots=None), dict(ldq=511), dict(ldqo=8), dict(ldk=64),
               dict(ldv=130)):
        assert call(**kw) == bad, kw
    for kw in (dict(q=addr(1, 4)), dict(qo=addr(2, 8)), dict(k=addr(3, 4)), dict(v=addr(4, 8)), dict(slots=addr(5, 2)),
               dict(pos=addr(0, 1)), dict(qg=addr(6, 8)), dict(kg=addr(6, 4))):
        assert call(**kw) == gq4.ERR_MISALIGNED, kw
    for kw in (dict(qo=addr(1, 256)), dict(qo=addr(1), ldqo=516), dict(qo=addr(3)), dict(slots=addr(22)), dict(k=addr(20, 64)),
               dict(qo=addr(23)), dict(qg=addr(2)), dict(inv=addr(21))):
        assert call(**kw) == gq4.ERR_ALIAS, kw
    assert call(T=0) == gq4.OK


@no_gpu_only
def test_tree_checks(gq4):
    def tree(B=2, T=8, words=1, window=0, sinks=0, **at):
        p = [at.get(n, addr(i)) for i, n in enumerate(["parents", "starts", "lens", "pos", "bits"])]
        return gq4.lib.gq4_kv_tree(B, T, words, window, sinks, *p, None)
    for kw in (dict(B=0), dict(B=65537), dict(T=-1), dict(words=0), dict(words=9), dict(window=-1), dict(sinks=-1),
               dict(parents=None), dict(starts=None), dict(lens=None), dict(pos=None), dict(bits=None)):
        assert tree(**kw) == gq4.ERR_INVALID_ARG, kw
    assert tree(bits=addr(4, 2)) == gq4.ERR_MISALIGNED
    assert tree(pos=addr(0, 4)) == gq4.ERR_ALIAS and tree(bits=addr(3)) == gq4.ERR_ALIAS
    assert tree(T=0) == gq4.OK


@no_gpu_only
def test_accept_checks(gq4):
    need = gq4.lib.gq4_kv_accept_workspace_bytes(4)
    assert need >= 16 and gq4.lib.gq4_kv_accept_workspace_bytes(0) == 0

    def accept(c=None, B=4, most=3, width=5, n_free=6, wb=need, **at):
        names = ["path", "counts", "starts", "lens", "table", "free", "count", "count_out", "lens_out", "ws"]
        p = [at.get(n, addr(i)) for i, n in enumerate(names)]
        return gq4.lib.gq4_kv_accept(B, most, width, n_free, ctypes.byref(c or cache(gq4)), *p, wb, None)
    bad = gq4.ERR_INVALID_ARG
    for kw in BAD_CACHES:
        assert accept(cache(gq4, **kw)) == bad, kw
    for kw in (dict(B=0), dict(B=65537, wb=1 << 20), dict(most=-1), dict(width=0), dict(n_free=-1), dict(width=1 << 28),
               dict(counts=None), dict(starts=None), dict(lens=None), dict(table=None), dict(free=None), dict(count=None),
               dict(count_out=None), dict(lens_out=None), dict(ws=None), dict(wb=need - 1)):
        assert accept(**kw) == bad, kw
    assert accept(path=addr(0, 2)) == gq4.ERR_MISALIGNED and accept(ws=addr(9, 16)) == gq4.ERR_MISALIGNED
    for kw in (dict(lens_out=addr(3, 4)), dict(count_out=addr(5, 8)), dict(free=addr(4, 16)), dict(ws=addr(8)),
               dict(free=addr(22, 64)), dict(path=addr(20, 32)), dict(lens_out=addr(1))):
        assert accept(**kw) == gq4.ERR_ALIAS, kw


def test_binding_refuses(gq4):
    x, i = torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int32)
    c = (torch.zeros(1, 2, 16, 8, dtype=torch.int32), torch.zeros(1, 2, 16, 2, 2)) * 2
    for call in (lambda: gq4.kv_rope_append(x, x, x, i, None, i, *c, 32), lambda: gq4.kv_tree(i, i, i, 1),
                 lambda: gq4.kv_accept(i, i, i, i, i, i, i, *c, 32)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_worked_path():
    """Two requests, pages of 16: nodes 0, 2, 5 of six behind 15 tokens; the first of twenty behind 3."""
    table, free = np.array([[4, 9], [2, 7]], np.int32), np.full(4, -1, np.int32)
    lens, free, count, moves, refused = M.accept(np.array([[0, 2, 5], [0, 0, 0]]), [3, 1], [0, 6, 26], [21, 23], table, free, 1,
                                                 10, 16)
    assert lens.tolist() == [18, 4] and moves == [(0, 17, 16), (0, 20, 17)] and not refused
    assert free.tolist() == [-1, 7, -1, -1] and count == 2
