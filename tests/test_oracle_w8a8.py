"""Pins of the W8A8 oracle (CPU)."""

from fractions import Fraction

import numpy as np

from oracle import hadamard as oh
from oracle import w8a8 as ow


def _round_half_even(f):
    n, r = f.numerator // f.denominator, f - f.numerator // f.denominator
    return n + (1 if r > Fraction(1, 2) or (r == Fraction(1, 2) and n % 2) else 0)


def test_codes_against_fractions():
    """Codes and scales of small rows, element by element in exact arithmetic on the float32 factors."""
    rng = np.random.default_rng(0)
    v = (rng.standard_normal((20, 48)) * np.exp(rng.uniform(-20, 20, (20, 1)))).astype(np.float32)
    v[3, :5] = [0.5, -0.5, 1.5, 2.5, 127]
    v[3, 5:] = 0
    q, s = ow.quantize_rows(v)
    for r in range(len(v)):
        amax = np.abs(v[r]).max()
        assert s[r] == np.float32(amax) / np.float32(127)
        inv = Fraction(float(np.float32(127) / amax))
        assert q[r].tolist() == [_round_half_even(Fraction(float(x)) * inv) for x in v[r]]
    assert q[3, :5].tolist() == [0, 0, 2, 2, 127]


def test_reconstruction_bound():
    rng = np.random.default_rng(1)
    v = (rng.standard_normal((50, 256)) * 3).astype(np.float32)
    q, s = ow.quantize_rows(v)
    err = np.abs(v - q.astype(np.float64) * s.astype(np.float64)[:, None])
    assert (err <= (0.5 + 2.0 ** -15) * s[:, None]).all() and np.abs(q).max() == 127


def test_special_rows():
    v = np.ones((5, 32), np.float32)
    v[0] = 0
    v[1] = 2.0 ** -101
    v[2, 3] = np.inf
    v[3, 4] = np.nan
    q, s = ow.quantize_rows(v)
    assert s[0] == 0 and s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3]) and s[4] == np.float32(1) / np.float32(127)
    assert (q[:4] == 0).all() and (q[4] == 127).all()


def test_butterflies_and_scale_fold():
    """The unnormalised butterflies times the normalisation are the block transform, and the rotated
    codes and scales stand for the rotated values."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((6, 256)).astype(np.float32)
    for B in (16, 32, 64, 128):
        assert np.array_equal(ow.butterflies(x, B) * oh.norm_const(B), oh.fwht_blocks(x, B))
        q, s = ow.quantize_act(x, None, B)
        r = oh.fwht_blocks(x, B)
        assert (np.abs(q.astype(np.float64) * s[:, None] - r) <= (0.5 + 2.0 ** -14) * s[:, None]).all()


def test_integer_layer():
    """Integer weights with unit scales on rows whose maximum is 127: the layer is the integer product."""
    rng = np.random.default_rng(3)
    x = rng.integers(-127, 128, (4, 64)).astype(np.float32)
    x[:, 0] = 127
    w = rng.integers(-128, 128, (7, 64)).astype(np.int8)
    y = ow.linear_f32(x, w, np.ones(7, np.float32), bias=np.full(7, 2.0, np.float32))
    assert np.array_equal(y, x.astype(np.int64) @ w.astype(np.int64).T + 2)


def test_rotation_cancels_in_the_product():
    """Weights and activations rotated and smoothed together: the 8-bit layer is near the plain one."""
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((8, 256)), rng.standard_normal((12, 256)) / 16
    lam = rng.uniform(0.5, 2, 256).astype(np.float32)
    for B in (0, 16, 128):
        qw, sw = ow.quantize_weight(w, lam, B)
        y = ow.linear_f32(x, qw, sw, lam, block=B)
        ref = x @ w.T
        assert np.linalg.norm(y - ref) <= 0.03 * np.linalg.norm(ref)
