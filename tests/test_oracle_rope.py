"""Pins of the norm + rotary oracle (CPU)."""

import cmath
import math

import numpy as np
import pytest

from oracle import rope


def test_against_complex_numbers():
    """A pure-Python loop over complex numbers, two axes, part of the head rotated."""
    rng = np.random.default_rng(0)
    x, pos, w = rng.standard_normal((3, 2, 12)), rng.integers(-9, 10, (3, 2)), rng.uniform(0.5, 2, 12)
    for layout in ("interleaved", "half", "axis_half"):
        for shared in (False, True):
            y, _ = rope.norm_rope(x, pos, [4, 6], w, 1e-6, 100.0, layout, shared)
            for t in range(3):
                for h in range(2):
                    r = 1 / math.sqrt(sum(v * v for v in x[t, h]) / 12 + float(np.float32(1e-6)))
                    u = [v * r * g for v, g in zip(x[t, h], w)]
                    want = list(u)
                    p = 0
                    for a, d in enumerate((4, 6)):
                        for i in range(d // 2):
                            base = (0, 4)[a]
                            e = {"interleaved": (2 * p, 2 * p + 1), "half": (p, p + 5),
                                 "axis_half": (base + i, base + i + d // 2)}[layout]
                            f = 100.0 ** (-2.0 * p / 10 if shared else -2.0 * i / d)
                            z = complex(u[e[0]], u[e[1]]) * cmath.exp(1j * float(pos[t, a]) * f)
                            want[e[0]], want[e[1]] = z.real, z.imag
                            p += 1
                    assert np.allclose(y[t, h], want, rtol=1e-13, atol=1e-13)


def test_rotation_keeps_norms_and_position_zero():
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((5, 3, 64)), rng.integers(0, 1000, (5, 3))
    y, u = rope.norm_rope(x, pos, [16, 24, 24])
    assert np.allclose((y * y).sum(-1), (u * u).sum(-1), rtol=1e-12)
    y0, u0 = rope.norm_rope(x, pos * 0, [16, 24, 24])
    assert np.array_equal(y0, u0)


@pytest.mark.parametrize("layout", ["interleaved", "half", "axis_half"])
def test_dot_products_depend_on_the_difference(layout):
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32))
    dots = []
    for shift in (0, 5, 1000):
        a, _ = rope.norm_rope(q, [[7 + shift, 3 + shift]], [16, 16], layout=layout)
        b, _ = rope.norm_rope(k, [[2 + shift, 9 + shift]], [16, 16], layout=layout)
        dots.append(float((a * b).sum()))
    assert np.allclose(dots, dots[0], rtol=1e-10)


def test_layouts_are_permutations_of_each_other():
    rng = np.random.default_rng(3)
    x, pos = rng.standard_normal((4, 2, 20)), rng.integers(0, 50, (4, 2))
    ref = rope.pair_table([8, 10], "interleaved", False)
    y, _ = rope.norm_rope(x, pos, [8, 10], norm=False)
    for layout in ("half", "axis_half"):
        tab = rope.pair_table([8, 10], layout, False)
        z = x.copy()
        for a, b in zip(ref, tab):
            z[..., b[0]], z[..., b[1]] = x[..., a[0]], x[..., a[1]]
        w, _ = rope.norm_rope(z, pos, [8, 10], norm=False, layout=layout)
        for a, b in zip(ref, tab):
            assert np.allclose(w[..., b[0]], y[..., a[0]]) and np.allclose(w[..., b[1]], y[..., a[1]])
    one = rope.pair_table([20], "half", False)
    assert one == rope.pair_table([20], "axis_half", False)


def test_far_angles_in_extended_precision():
    """Exponents that are no float64 (2 i / 40) and angles of about 1e12 against 60 digits: what extended precision loses
    is the exponent's rounding times ln(theta) (15 * 2^-64), a power (2^-63) and a product (2^-64), below 20 * 2^-64."""
    from decimal import Decimal as Dec, getcontext
    getcontext().prec = 60
    pi = Dec("3.14159265358979323846264338327950288419716939937510582097494")
    for theta, pos in ((3e-7, 1234567), (1e4, 10 ** 12 + 39)):
        x = np.zeros((1, 1, 40))
        x[..., ::2] = 1.0
        y, _ = rope.norm_rope(x, [[pos]], [40], theta=theta, norm=False)
        for i in range(20):
            angle = Dec(pos) * (-(Dec(theta).ln() * Dec(2 * i) / Dec(40))).exp()
            r = float(angle % (2 * pi))
            tol = float(angle) * 20 * 2.0 ** -64 + 4 * 2.0 ** -53 * 7
            assert abs(y[0, 0, 2 * i] - math.cos(r)) < tol and abs(y[0, 0, 2 * i + 1] - math.sin(r)) < tol, (theta, i)
