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
