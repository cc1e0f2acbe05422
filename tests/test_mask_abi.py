"""Refusals of the attention with masks on the host (made-up device addresses, every call invalid, nothing launched), the
struct's layout, and worked examples of the restatements."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from tests import mask_ref as M
from tests.gpu_util import gq4_module
from tests.test_abi import ROOT, addr, no_gpu_only
from tests.test_kv_abi import cache


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
    need = gq4.kv_attention_workspace_bytes(4, 8, 2, 64)
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
