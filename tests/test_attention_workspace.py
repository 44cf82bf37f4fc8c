"""The attentions' workspace stays in proportion to what the GPU holds, whatever the batch and max_q (CPU: sizes only)."""

import ctypes
import os
import random

import pytest

import w4a4_bit_quantized_amd as w4
from test_cache_abi import cache, lib  # noqa: F401
from w4a4_bit_quantized_amd import binding

pytestmark = pytest.mark.skipif(bool(os.environ.get("W4A4_LIBRARY")), reason="a host-only build: no kernels, no workspace")


def need(lib, T, B, H, heads, D, mq):
    a = binding.Attention(None, H * D, D, None, H * D, D, T, H, None, 0, 0, None, 1, B, mq, 0, 0, 1.0, D, 0)
    return lib.w4a4_attention_workspace_bytes(ctypes.byref(a), ctypes.byref(cache(heads=heads, D=D)))


def wide(D):
    return 64 if D <= 64 else 128 if D <= 128 else 256


def bound(D):
    """Eight times the workgroups that the GPU holds, each with a tile of 128 rows in float32.  With R rows and at least S
    sequences of max_q queries, tiles are counted as W = (R / 128 + (S + 1) / 2) heads, and cut into P pieces with P W <= 4/3 of the
    workgroups (P >= 2).  Slots are at most 6 W: min(R / 128 + batch, 5 R / 128) with rows_from = 32, R / 128 + 16 / heads where
    that is 16, R / 128 + 2 S where the tiles take all sequences."""
    return 8 * (512 if D <= 128 else 256) * 128 * (2 + wide(D)) * 4


def test_short_sequences_among_long_ones(lib):
    # a piece of 256 queries among 255 single tokens; single tokens with max_q left at the number of tokens
    for T, B, H, heads, D, mq in ((511, 256, 32, 8, 128, 256), (256, 256, 32, 8, 128, 256), (512, 512, 32, 8, 128, 512),
                                  (1024, 1024, 8, 8, 128, 1024), (4095, 4000, 64, 4, 256, 96), (1 << 20, 1 << 20, 8, 8, 64, 1 << 20)):
        assert 0 < need(lib, T, B, H, heads, D, mq) <= bound(D), (T, B, H, heads, D, mq)


def test_any_shape(lib):
    rng = random.Random(2)
    for _ in range(20000):
        D, heads = rng.choice([64, 72, 128, 256]), rng.choice([1, 2, 4, 8, 16, 64])
        H = heads * rng.choice([1, 2, 4, 5, 7, 8, 16, 64])
        T, B = (int(2 ** rng.uniform(0, 17)) for _ in range(2))
        mq = min(T, rng.choice([T, max(1, T // B), int(2 ** rng.uniform(0, 17))]))
        if T * H <= 1 << 30:
            assert 0 < need(lib, T, B, H, heads, D, mq) <= bound(D), (T, B, H, heads, D, mq)


def tensors(T=6, H=4, heads=2, D=64, dtype=None):
    import torch
    dtype = dtype or torch.bfloat16
    return torch.zeros(T, H, D, dtype=dtype), *(torch.zeros(8, 16, heads, D, dtype=dtype) for _ in range(2))


def test_helper_gives_what_the_call_asks_for(lib):
    t = tensors(T=256, H=32, heads=8, D=128)
    size = lambda *args, **kw: w4.attention_workspace_bytes(*t, *args, **kw)
    assert size(256) == need(lib, 256, 256, 32, 8, 128, 256) > 4 * size(256, uniform=True)
    assert size(256, uniform=True) == size(256, 1) == size(256, 1, uniform=True) == need(lib, 256, 256, 32, 8, 128, 1)
    assert size(2, uniform=True) == size(2, 128) and size(256, 2 ** 80) == size(256)
    for args, kw in (((3,), dict(uniform=True)), ((0,), dict(uniform=True)), ((2, 100), dict(uniform=True)), ((-1,), {}), ((256, -1), {}),
                     ((2 ** 64 + 256,), {}), ((5 - 2 ** 64,), {}), ((2 ** 30 + 1,), {}), ((256, 5 - 2 ** 64), {})):
        with pytest.raises(ValueError):
            size(*args, **kw)


def test_helper_refuses_what_the_call_refuses(lib):
    import torch
    q, k, v = tensors()
    for bad in ((q[..., :32], k, v), (q, k[..., :60], v[..., :60]), (q[:, :3], k, v), (q, k[:, :, :0], v[:, :, :0]),
                tensors(D=60), tensors(D=264), (torch.zeros(6, 4, 68, dtype=q.dtype)[..., 2:66].as_strided((6, 4, 64), (270, 66, 1)), k, v)):
        with pytest.raises(ValueError):
            w4.attention_workspace_bytes(*bad, 2)
    with pytest.raises((TypeError, ValueError)):
        w4.attention_workspace_bytes(*tensors(dtype=torch.float32), 2)
    assert w4.attention_workspace_bytes(*tensors(T=0), 2) > 0 and w4.attention_workspace_bytes(*tensors(T=0), 0, uniform=True) > 0


def test_uniform_batches_need_no_more_than_others(lib):
    """A workspace for a call with q_starts and the default max_q holds the same batch without them."""
    rng = random.Random(3)
    for _ in range(20000):
        D, heads = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8, 16])
        H = heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        B, each = int(2 ** rng.uniform(0, 11)), int(2 ** rng.uniform(0, 9))
        assert need(lib, B * each, B, H, heads, D, each) <= need(lib, B * each, B, H, heads, D, B * each), (B, each, H, heads, D)
