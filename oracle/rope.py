"""RMS norm of q / k heads with the multi-axis rotary rotation (oracle, test infrastructure only),
in float64 with the angles in extended precision.

``pair_table`` lists, for every rotated pair, its two elements, its axis and its frequency exponent;
``norm_rope`` applies norm, weight and rotation.

Pins (``tests/test_oracle_rope.py``): a pure-Python complex-number loop, norms kept by the rotation,
relative-position invariance of dot products, position 0 as the identity, and the agreement of the
layouts under the permutations that relate them.
"""

import numpy as np


def pair_table(axis_dims, layout, shared):
    """[(e0, e1, axis, exponent)] of every pair; the pair turns by pos[axis] * theta^-exponent.  (The exponents in
    extended precision too: rounded to float64, 2 i / 40 moves the angle by up to ln(theta) 2^-54 of itself.)"""
    rot = sum(axis_dims)
    out = []
    base = 0
    for a, d in enumerate(axis_dims):
        for i in range(d // 2):
            p = base // 2 + i
            e0, e1 = {"interleaved": (2 * p, 2 * p + 1), "half": (p, p + rot // 2),
                      "axis_half": (base + i, base + i + d // 2)}[layout]
            out.append((e0, e1, a, np.longdouble(2 * p) / rot if shared else np.longdouble(2 * i) / d))
        base += d
    return out


def norm_rope(x, positions, axis_dims, weight=None, eps=1e-6, theta=10000.0, layout="interleaved", shared=False,
              norm=True):
    """x (T, H, D) -> (y float64, u float64): the result, and the normed values before the rotation."""
    u = np.asarray(x, np.float64)
    if norm:
        u = u / np.sqrt((u * u).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
        if weight is not None:
            u = u * np.asarray(weight, np.float64)
    y = u.copy()
    table = pair_table(axis_dims, layout, shared)
    if table:
        e0 = [t[0] for t in table]
        e1 = [t[1] for t in table]
        pos = np.asarray(positions).reshape(len(u), len(axis_dims)).astype(np.longdouble)
        freq = np.array([np.longdouble(theta) ** -t[3] for t in table], np.longdouble)
        ang = pos[:, [t[2] for t in table]] * freq[None, :]
        c = np.cos(ang).astype(np.float64)[:, None, :]
        s = np.sin(ang).astype(np.float64)[:, None, :]
        y[..., e0] = u[..., e0] * c - u[..., e1] * s
        y[..., e1] = u[..., e0] * s + u[..., e1] * c
    return y, u
