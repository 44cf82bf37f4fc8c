"""Pins of the attention oracle (CPU)."""

import math

import numpy as np

from oracle import attention as oa


def draw(seed, n, l, H, Hk, D):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((n, H, D)), rng.standard_normal((l, Hk, D)), rng.standard_normal((l, Hk, D))


def test_against_a_loop_over_single_keys():
    n, l, H, Hk, D = 3, 7, 4, 2, 4
    q, k, v = draw(0, n, l, H, Hk, D)
    mask = np.array([[1, 0, 0], [1, 1, 0], [1, 0, 1]], bool)
    pos = np.array([4, 5, 5])
    for window, sinks, m, p in ((0, 0, None, None), (3, 0, None, None), (2, 1, None, None), (0, 0, mask, None), (3, 1, mask, pos)):
        out = oa.attend(q, k, v, oa.visible(n, l, window, sinks, m, p), 0.5)[0]
        for i in range(n):
            for h in range(H):
                at = l - n + i if m is None else 10 ** 9 if p is None else int(p[i])
                num, den = [0.0] * D, 0.0
                for j in range(l):
                    if m is not None and j >= l - n:
                        see = m[i, j - (l - n)]
                    else:
                        see = j <= at and (window == 0 or at - j < window or j < sinks)
                    if see:
                        w = math.exp(0.5 * sum(float(a) * float(b) for a, b in zip(q[i, h], k[j, h // 2])))
                        den += w
                        num = [x + w * float(y) for x, y in zip(num, v[j, h // 2])]
                assert np.allclose(out[i, h], np.array(num) / den, rtol=1e-12, atol=1e-13)


def test_equal_keys_and_single_keys():
    q, k, v = draw(1, 2, 9, 2, 1, 8)
    k[:] = k[0]
    seen = oa.visible(2, 9)
    out = oa.attend(q, k, v, seen, 1.0)[0]
    assert np.allclose(out[0, 0], v[:8, 0].mean(0)) and np.allclose(out[1, 1], v[:, 0].mean(0))
    one = oa.attend(q, k, v, oa.visible(2, 9, window=1), 1.0)[0]
    assert np.allclose(one[0, 0], v[7, 0]) and np.allclose(one[1, 0], v[8, 0])
    assert not oa.attend(q, k, v, np.zeros((2, 9), bool), 1.0)[0].any()


def test_masks_that_say_the_same():
    causal = oa.visible(5, 12)
    assert (oa.visible(5, 12, window=12) == causal).all() and (oa.visible(5, 12, 3, 12) == causal).all()
    assert (oa.visible(5, 12, mask=np.tril(np.ones((5, 5), bool))) == causal).all()
    assert (oa.visible(5, 12, 4, 2, np.tril(np.ones((5, 5), bool)), np.arange(7, 12))[:, :7] == oa.visible(5, 12, 4, 2)[:, :7]).all()
    assert oa.visible(4, 2).sum() == 1 + 2  # more queries than keys: the first see nothing
    assert oa.visible(1, 0).shape == (1, 0)


def test_order_of_pages():
    q, k, v = draw(2, 4, 11, 2, 2, 8)
    rng = np.random.default_rng(3)
    outs = []
    for order in (np.arange(6), rng.permutation(6)):
        kc, vc = np.full((6, 2, 2, 8), np.nan), np.full((6, 2, 2, 8), np.nan)
        table = order[None, :6].astype(np.int32)
        for j in range(11):
            kc[order[j // 2], j % 2], vc[order[j // 2], j % 2] = k[j], v[j]
        outs.append(oa.paged(q, kc, vc, table, [11], [0, 4], 0.3)[0])
    assert np.array_equal(*outs)
    assert np.allclose(outs[0], oa.attend(q, k, v, oa.visible(4, 11), 0.3)[0])
