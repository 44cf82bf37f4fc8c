"""GPU tests of attention at its limits (needs an MI355X): see test_gpu_attention.py for the batches and their bounds."""

import numpy as np
import pytest

from test_gpu_attention import DTYPES, Batch, w4  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 50])
def test_a_pool_of_no_pages(w4, n):
    """Whatever the lengths say, nothing is seen: zeros."""
    b = Batch(1, [(n, 90), (n, 200)], 4, 2, 64, 16, "bf16")
    out = w4.paged_attention(b.dq, b.dk[:0], b.dv[:0], b.dt, b.dl)
    assert out.shape == b.dq.shape and (out == 0).all()
    m, pos = b.tree()
    b.dk, b.dv = b.dk[:0], b.dv[:0]
    assert (b.run_tree(w4, m, pos, window=9, sinks=2) == 0).all()


@pytest.mark.parametrize("big", [5 - 2 ** 64, -2 ** 63 - 1, 2 ** 63, 2 ** 64 + 5])
def test_numbers_past_64_bits(w4, big):
    """Refused, also below zero: their lower 64 bits may be a window."""
    b = Batch(2, [(1, 90)], 4, 2, 64, 16, "bf16")
    for kw in (dict(window=big), dict(window=9, sinks=big)):
        with pytest.raises(ValueError, match="out of range"):
            b.run(w4, **kw)
    with pytest.raises(w4.W4A4Error, match="SHAPE"):
        b.run(w4, window=-2 ** 63)
