"""Pins of the oracle's norm with rotation (against differences and closed forms) and of its 4-bit rows."""
import numpy as np
import pytest

import oracle
from oracle import paged


def tables(n, half, base=10000.0):
    a = np.arange(n)[:, None] * base ** (-np.arange(half) / half)
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("half", [0, 8, 32])
@pytest.mark.parametrize("norm", [False, True])
def test_gradient_against_differences(interleaved, half, norm):
    r = np.random.default_rng(3)
    T, heads, d = 3, 2, 64
    x, w = r.standard_normal((T, heads, d)), 1 + 0.3 * r.standard_normal(d)
    pos = np.array([5, 0, 11])
    cos, sin = tables(12, half) if half else (None, None)
    kw = dict(w=w if norm else None, eps=1e-3, norm=norm, cos=cos, sin=sin, interleaved=interleaved)
    dy = r.standard_normal(x.shape)

    def loss(x, w):
        return float((oracle.norm_rope(x, pos, **dict(kw, w=w if norm else None)) * dy).sum())

    dx, dw = oracle.norm_rope_backward(x, dy, pos, **kw)
    h = 1e-5   # central differences: h^2 f''' / 6 plus 2^-52 |f| / h, both below 1e-8 of the values here
    for idx in [(0, 0, 0), (1, 1, 7), (2, 0, 33), (2, 1, 63)]:
        e = np.zeros_like(x)
        e[idx] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[idx]) < 1e-7
    if norm:
        for j in (0, 31, 63):
            e = np.zeros(d)
            e[j] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[j]) < 1e-7


def test_rotation_keeps_lengths_and_relative_angles():
    r = np.random.default_rng(4)
    cos, sin = tables(200, 32)
    q, k = r.standard_normal((1, 1, 64)), r.standard_normal((1, 1, 64))
    for il in (False, True):
        def at(x, p):
            return oracle.norm_rope(x, [p], norm=False, cos=cos, sin=sin, interleaved=il)[0, 0]
        assert np.linalg.norm(at(q, 77)) == pytest.approx(np.linalg.norm(q), rel=1e-14)
        assert at(q, 150) @ at(k, 120) == pytest.approx(at(q, 50) @ at(k, 20), rel=1e-12)   # distance alone
        # float32 steps agree with the matrix form to a few roundings of the pair's length
        y = paged.turn_f32(q, cos[[77]], sin[[77]], il)[0, 0]
        assert np.abs(y - at(np.float32(q), 77)).max() <= 4 * 2.0 ** -24 * 2 * np.abs(q).max()


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(5).standard_normal((4, 3, 128)) * 7
    y = oracle.norm_rope(x, [0, 1, 2, 3], eps=0.0)
    assert np.allclose((y * y).mean(-1), 1, rtol=1e-14)


def rows():
    r = np.random.default_rng(6)
    x = r.standard_normal((9, 128)).astype(np.float32)
    x[1] *= 1e-30
    x[2] *= 1e30
    x[3] = 100 + 0.01 * x[3]        # far from 0: the floor of the scale is not reached, zero carries it
    x[4] = -5.0                     # constant
    x[5] = 0.0
    x[6, :64] = 1e9                 # constant and large beside an ordinary group
    x[7, 0] = 300.0                 # outlier
    return paged.bf16_nearest(x)


def test_quantisation_error_is_half_a_step():
    x = rows()
    codes, scale, zero = paged.quantise(x)
    assert codes.max() <= 15
    assert np.all(scale > 0) and np.all(np.isfinite(scale)) and np.all(np.isfinite(zero))
    # scales and zeros are bf16
    assert np.array_equal(paged.bf16_nearest(scale), scale) and np.array_equal(paged.bf16_nearest(zero), zero)
    err = np.abs(paged.values(codes, scale, zero) - x).reshape(9, 2, 64)
    # (x - zero) and the quotient are rounded to 24 bits: 15 codes times two roundings of 2^-24
    assert np.all(err <= scale[..., None] * (0.5 + 15 * 2.0 ** -23))
    # the range reaches both ends of the group: no value is clipped, and no code range is left over
    spread = x.reshape(9, 2, 64).max(-1) - x.reshape(9, 2, 64).min(-1)
    # (where scale is above its floor: with spread < 15 2^-100 the greatest code is spread / 2^-100 < 15)
    wide = (spread > 2.0 ** -8 * np.abs(x.reshape(9, 2, 64)).max(-1)) & (spread >= 15 * 2.0 ** -100)
    assert np.all(codes.reshape(9, 2, 64).max(-1)[wide] >= 14)


def test_directed_rounding():
    x = np.float32([1.0, 1.0000001, -1.0000001, 0.0, -0.0, 3.1415927, -3.1415927, 1e-40])
    lo, hi = paged.bf16_toward(x, False), paged.bf16_toward(x, True)
    assert np.all(lo <= x) and np.all(hi >= x)
    assert np.all((lo == hi) == (paged.bf16_nearest(x) == x))


def test_pack_puts_even_dims_low():
    codes = np.arange(16, dtype=np.uint8)
    assert paged.pack(codes)[:3].tolist() == [0x10, 0x32, 0x54]


def test_attention_paged_is_attention():
    r = np.random.default_rng(7)
    q = r.standard_normal((2, 3, 4, 64))
    keys = [r.standard_normal((n, 2, 64)) for n in (5, 2)]
    vals = [r.standard_normal((n, 2, 64)) for n in (5, 2)]
    o, lse = oracle.paged.attention_paged(q, keys, vals, 0.125, True)
    assert np.isneginf(lse[1, :, 0]).all() and np.all(o[1, 0] == 0)     # 2 keys, 3 queries: the first sees none
    s = 0.125 * keys[0][:4, 1] @ q[0, 1, 3]
    p = np.exp(s) / np.exp(s).sum()
    assert np.allclose(o[0, 1, 3], p @ vals[0][:4, 1], rtol=1e-12) and lse[0, 3, 1] == pytest.approx(np.log(np.exp(s).sum()))
