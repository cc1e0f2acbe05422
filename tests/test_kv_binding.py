"""The binding of the cache calls on the host: what it asks torch for."""

import pytest
import torch

from tests.gpu_util import gq4_module


@pytest.mark.parametrize("device,want", [(0, 0), (1, 1), (None, "cuda"), ("cuda:1", "cuda:1")])
def test_cache_device(monkeypatch, device, want):
    """Device 0 by its number is device 0, not whichever is current."""
    gq4 = gq4_module()
    asked = []
    monkeypatch.setattr(gq4.torch, "zeros", lambda *a, device=None, **kw: asked.append(device))
    gq4.kv_cache(1, 1, 16, 64, 32, device=device)
    assert asked == [want] * 4
