"""GPU tests of rotation and append for keys whose size is far from 1, against 64 bits."""

import numpy as np
import pytest
import torch

from int4_group_quantized_quant_gb300 import inputs as I
from tests import kv_ref as R
from tests.gpu_util import dev, gq4_module, host, requires_cuda
from tests.test_gpu_trees import codes_of, inv_freq

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def gq4():
    g = gq4_module()
    g.device_error(clear=True)
    return g


def turned_back(y, pos, inv, inter):
    """The rows that the rotation turns into y, in 64 bits."""
    x, rot = y.copy(), 2 * len(inv)
    ang = pos[:, None].astype(np.float64) * inv.astype(np.float64)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    x[..., a], x[..., b] = y[..., a] * c + y[..., b] * s, y[..., b] * c - y[..., a] * s
    return x


def border_rows(g, T, KH, D, gs):
    """Groups from -7/8 to 1 whose values between are halves between two codes."""
    y = g.integers(0, 15, (T, KH, D // gs, gs)) + 0.5
    y[..., 0], y[..., -1] = 0, 15
    return (y - 7).reshape(T, KH, D) / 8


def append(gq4, k, pos, inv, inter, gain, eps, gs, page=16):
    """The keys' codes and scales [T, KH, ...] as one call leaves them."""
    T, KH, D = k.shape
    cache = gq4.kv_cache((T + page - 1) // page, KH, page, D, gs)
    slots = np.arange(T, dtype=np.int32)
    gq4.kv_rope_append(None, dev(k), dev(np.zeros_like(k)), dev(pos), dev(inv), dev(slots), *cache, gs, interleaved=inter,
                       k_gain=None if gain is None else dev(gain), eps=eps)
    codes, sz = codes_of([host(t) for t in cache], slots, page)
    return codes[0], sz[0]


def check(codes, sz, y, size, gs):
    """Codes exactly; what they stand for within 64 units of 2^-24 of the largest pair of the row, as
    test_gpu_trees.check_rows derives."""
    want, want_sz = R.quantise(y.astype(np.float32), gs)
    assert np.array_equal(codes, want)
    err = np.abs(R.values(codes, sz) - R.values(want, want_sz))
    assert np.all(err <= 64 * 2.0 ** -24 * size.max(-1, keepdims=True))


SHAPES = [(128, 32, 128, False), (256, 64, 128, True), (96, 96, 96, False), (64, 32, 32, True)]


@pytest.mark.parametrize("power", [-110, -75, -62, -49, -30, 30, 49, 62, 75, 110])
@pytest.mark.parametrize("D,gs,rot,inter", SHAPES)
def test_normalised_keys_of_any_size(gq4, D, gs, rot, inter, power):
    """Without eps a row's size falls out of the norm, also where the squares are 0 or infinite as f32: codes next to a
    border are those of the row in 64 bits, and no row is zero or not finite."""
    T, KH = 120, 3
    g = I.rng(2600, D, gs, rot)
    inv, pos = inv_freq(rot), g.integers(0, 50000, T).astype(np.int32)
    gain = np.exp2(g.integers(-1, 2, D)).astype(np.float32)
    k = (turned_back(border_rows(g, T, KH, D, gs), pos, inv, inter) / gain * 2.0 ** power).astype(np.float32)
    k[1] *= 2.0 ** (-power)                # one row of ordinary size among them
    codes, sz = append(gq4, k, pos, inv, inter, gain, 0.0, gs)
    assert gq4.device_error(clear=True) == 0
    y, size = R.norm_rope(k, gain, 0.0, pos, inv, inter)
    check(codes, sz, y, size, gs)


def test_normalised_rows_of_huge_and_not_finite_values(gq4):
    """A row of f32's largest values with eps; an infinity and a NaN spoil their row's groups as the formula does, a row of
    zeros without eps is 0 / 0."""
    T, KH, D, gs = 6, 2, 64, 32
    g = I.rng(2601)
    k = g.standard_normal((T, KH, D)).astype(np.float32)
    k[0] = np.where(k[0] > 0, np.float32(3.4e38), np.float32(-3.4e38))
    k[2, 0, 5], k[3, 1, 40], k[4, 0] = np.inf, np.nan, 0
    pos, inv, gain = np.arange(T, dtype=np.int32), inv_freq(16), np.ones(D, np.float32)
    codes, sz = append(gq4, k, pos, inv, False, gain, 0.0, gs)
    assert gq4.device_error(clear=True) == 1 << 3
    with np.errstate(all="ignore"):
        y, size = R.norm_rope(k, gain, 0.0, pos, inv, False)
        y[2, 0, 32:] = 0                   # finite over infinite
    bad = ~np.isfinite(y.reshape(T, KH, D // gs, gs)).all(-1)
    assert bad[2, 0].tolist() == [True, False] and bad[3, 1].all() and bad[4, 0].all() and bad.sum() == 5
    assert np.array_equal(np.isnan(sz).all(-1), bad) and np.array_equal(np.isnan(sz).any(-1), bad)
    good = ~bad.any(-1)
    want, want_sz = R.quantise(y.astype(np.float32), gs)
    assert np.array_equal(codes[good], want[good])
    err = np.abs(R.values(codes, sz) - R.values(want, want_sz))[good]
    assert np.all(err <= 64 * 2.0 ** -24 * size[good].max(-1, keepdims=True))
    # with eps nothing changes for the large row, and zeros stay zeros
    codes, sz = append(gq4, k[[0, 4]], pos[[0, 4]], inv, False, gain, 1e-6, gs)
    y, size = R.norm_rope(k[[0, 4]], gain, 1e-6, pos[[0, 4]], inv, False)
    check(codes, sz, y, size, gs)
    assert np.array_equal(sz[1, 0], [[1, 0], [1, 0]]) and gq4.device_error(clear=True) == 0


@pytest.mark.parametrize("norm", [False, True])
def test_small_groups_next_to_a_border(gq4, norm):
    """Groups of some 2^-60 to 2^-118 beside one of ordinary size: their codes are those of 64 bits as well."""
    T, KH, D, gs = 400, 4, 128, 32
    g = I.rng(2602, norm)
    inv, pos = inv_freq(D), g.integers(0, 50000, T).astype(np.int32)
    small = np.exp2([0.0, -60.0, -100.0, -118.0]).repeat(gs).astype(np.float32)
    y = border_rows(g, T, KH, D, gs)
    x = turned_back(y, pos, inv, True)     # (pairs of neighbours: of one group)
    # by the row or by the gains
    k, gain = (x.astype(np.float32), small) if norm else ((x * small).astype(np.float32), None)
    codes, sz = append(gq4, k, pos, inv, True, gain, 1e-6, gs)
    assert gq4.device_error(clear=True) == 0
    y, _ = R.norm_rope(k, gain, 1e-6, pos, inv, True)
    want, _ = R.quantise(y.astype(np.float32), gs)
    wrong = (codes != want).reshape(T * KH, D // gs, gs).sum((0, 2))
    assert wrong.tolist() == [0, 0, 0, 0]
