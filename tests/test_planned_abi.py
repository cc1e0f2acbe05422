"""Refusals of the calls that take the planned slots, on the host (made-up device addresses, every call invalid, nothing
launched)."""

import ctypes

import pytest
import torch

from tests.gpu_util import gq4_module
from tests.test_abi import addr, no_gpu_only
from tests.test_kv_abi import BAD_CACHES, cache


@pytest.fixture(scope="module")
def gq4():
    return gq4_module()


@no_gpu_only
def test_tree_checks(gq4):
    def tree(B=2, T=8, words=1, window=0, sinks=0, **at):
        p = [at.get(n, addr(i)) for i, n in enumerate(["parents", "slots", "starts", "lens", "pos", "bits"])]
        return gq4.lib.gq4_kv_tree_planned(B, T, words, window, sinks, *p, None)
    for kw in (dict(B=0), dict(B=65537), dict(T=-1), dict(words=0), dict(words=9), dict(window=-1), dict(sinks=-1),
               dict(parents=None), dict(slots=None), dict(starts=None), dict(lens=None), dict(pos=None), dict(bits=None)):
        assert tree(**kw) == gq4.ERR_INVALID_ARG, kw
    assert tree(bits=addr(5, 2)) == gq4.ERR_MISALIGNED and tree(slots=addr(1, 2)) == gq4.ERR_MISALIGNED
    assert tree(pos=addr(1, 4)) == gq4.ERR_ALIAS and tree(bits=addr(1)) == gq4.ERR_ALIAS
    assert tree(T=0) == gq4.OK


@no_gpu_only
def test_accept_checks(gq4):
    need = gq4.lib.gq4_kv_accept_workspace_bytes(4)

    def accept(c=None, B=4, T=9, most=3, width=5, n_free=6, wb=need, **at):
        names = ["path", "counts", "slots", "starts", "lens", "table", "free", "count", "count_out", "lens_out", "ws"]
        p = [at.get(n, addr(i)) for i, n in enumerate(names)]
        return gq4.lib.gq4_kv_accept_planned(B, T, most, width, n_free, ctypes.byref(c or cache(gq4)), *p, wb, None)
    bad = gq4.ERR_INVALID_ARG
    for kw in BAD_CACHES:
        assert accept(cache(gq4, **kw)) == bad, kw
    for kw in (dict(B=0), dict(B=65537, wb=1 << 20), dict(T=-1), dict(most=-1), dict(width=0), dict(n_free=-1),
               dict(width=1 << 28), dict(counts=None), dict(slots=None), dict(starts=None), dict(lens=None), dict(table=None),
               dict(free=None), dict(count=None), dict(count_out=None), dict(lens_out=None), dict(ws=None), dict(wb=need - 1)):
        assert accept(**kw) == bad, kw
    for kw in (dict(path=addr(0, 2)), dict(slots=addr(2, 1)), dict(ws=addr(10, 16))):
        assert accept(**kw) == gq4.ERR_MISALIGNED, kw
    for kw in (dict(lens_out=addr(4, 4)), dict(count_out=addr(6, 8)), dict(free=addr(5, 16)), dict(ws=addr(9)),
               dict(free=addr(22, 64)), dict(slots=addr(20, 32)), dict(slots=addr(9, 8)), dict(lens_out=addr(2))):
        assert accept(**kw) == gq4.ERR_ALIAS, kw


def test_binding_refuses(gq4):
    i = torch.zeros(2, dtype=torch.int32)
    c = (torch.zeros(1, 2, 16, 8, dtype=torch.int32), torch.zeros(1, 2, 16, 2, 2)) * 2
    for call in (lambda: gq4.kv_tree(i, i, i, 1, slots=i), lambda: gq4.kv_accept(i, i, i, i, i, i, i, *c, 32, slots=i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
