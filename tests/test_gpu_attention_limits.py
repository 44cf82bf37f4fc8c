"""GPU tests of attention at its limits (needs an MI355X): see test_gpu_attention.py for the batches and their bounds."""

import numpy as np
import pytest

from oracle import hadamard as oh
from test_gpu_attention import DTYPES, HALF, TINY, Batch, w4  # noqa: F401
from test_gpu_w8a8 import dev, host

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


def sums_limit(res, dtype, D, keys):
    """The bound of test_gpu_attention.py's head, A (h + 2 e) and the output's half step, for both kernels: the sums below the
    fraction are of float32 probabilities (in the tiles 16 pairs of each 64 keys first, and one addition to the running sum: less
    than the 32 + B there).  The reference of these rows is set by their first block and raised by none (no score passes it by
    2^8): two factors instead of one per block, with the join's.  In f16 a probability of less than 2^-21 of the row's
    reference is off by 2^-32 of it."""
    o, absolute, spread, small = res
    blocks = keys / 32 + 1
    e = (D + 4) * 2.0 ** -23 * spread + 3 * (2.0 ** -21 + 2.0 ** -23 * spread) + 2.0 ** -23 * (blocks + 32)
    err = absolute * (HALF[dtype] + 2 * e[..., None])
    if dtype == "f16":
        err = err + 2.0 ** -32 * small
    return err + (np.abs(o) + err) * HALF[dtype] + TINY[dtype]


def one_head(w4, n, scores, v, dtype, D=64):
    """The last n queries of one head over keys of these scores (sums of three elements of each key) and values (keys, D): the
    kernel's rows, and the oracle's with its bounds."""
    l = len(scores)
    b = Batch(20, [(n, l)], 1, 1, D, 16, dtype, poison=0.0)
    k = np.zeros((l, D), np.float32)
    rest = np.asarray(scores, np.float64)
    for c in range(3):
        k[:, c] = oh.to_f32(oh.from_f32(rest.astype(np.float32), dtype), dtype)
        rest = rest - k[:, c]
    j = np.arange(l)
    for name, x in (("kc", k), ("vc", v)):
        pool = oh.to_f32(getattr(b, name), dtype).copy()
        pool[b.table[0, j // 16], j % 16, 0] = x
        setattr(b, name, oh.from_f32(pool.astype(np.float32), dtype))
    q = np.zeros((n, 1, D), np.float32)
    q[:, :, :3] = 1.0
    b.q = oh.from_f32(q, dtype)
    b.dq, b.dk, b.dv = (dev(x, dtype) for x in (b.q, b.kc, b.vc))
    got = oh.to_f32(host(b.run(w4, scale=1.0)), dtype).astype(np.float64)
    return got, b.expected(scale=1.0)


def within(got, res, dtype, keys, what, D=64):
    off = ~(np.abs(got - res[0]) <= sums_limit(res, dtype, D, keys))
    at = np.argwhere(off)
    assert at.size == 0, (f"{what}: {len(at)} of {off.size} off, first {at[:3].tolist()}: {got[tuple(at[0])]} for "
                          f"{res[0][tuple(at[0])]}, allowed {sums_limit(res, dtype, D, keys)[tuple(at[0])]}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 70], ids=["stream", "tiles"])
def test_many_small_probabilities(w4, n, dtype):
    """One strong first key, as a sink is, and tens of thousands far below it, whose probabilities are subnormal in f16 or less
    than its smallest and together matter."""
    l = 30000
    for below in (9.0, 10.5, 13.0, 16.0, 17.4, 18.5):
        print(f"\n{n} {dtype} {below}", flush=True)
        scores = np.full(l, -below)
        scores[0] = 0.0
        v = np.ones((l, 64)) * np.linspace(0.5, 1.5, 64)
        v[0] = 0.0
        got, res = one_head(w4, n, scores, v, dtype)
        assert (res[0][0, 0] > 2.0 ** -14).all()
        within(got, res, dtype, l, f"{below} below")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 70], ids=["stream", "tiles"])
def test_small_probabilities_of_one_reference(w4, n, dtype):
    """The same in a batch of so many heads that no row's keys are cut into pieces, which would have references of their own:
    32 sequences on the same pages, of 64 heads."""
    D, l, heads, page, B = 64, 2048, 64, 16, 32
    print(f"\n{n} {dtype}", flush=True)
    b = Batch(22, [(n, l)], heads, heads, D, page, dtype)
    k = np.zeros((b.pages, page, heads, D), np.float32)
    j = np.arange(l)
    low = -np.tile([9.0, 12.0, 15.0, 16.0, 17.0, 17.4, 18.0, 19.0], heads // 8).astype(np.float32)
    k[b.table[0, j // page], j % page, :, 0] = low - 0.125 * (j % 4)[:, None].astype(np.float32)
    k[b.table[0, 0], 0, :, 0] = 0.0
    v = np.zeros_like(k)
    v[b.table[0, j // page], j % page] = 100.0 * np.linspace(0.5, 1.5, D)
    v[b.table[0, 0], 0] = 0.0
    q = np.zeros((n, heads, D), np.float32)
    q[..., 0] = 1.0
    b.q, b.kc, b.vc = (oh.from_f32(x, dtype) for x in (q, k, v))
    res = b.expected(scale=1.0)
    got = w4.paged_attention(dev(np.tile(b.q, (B, 1, 1)), dtype), dev(b.kc, dtype), dev(b.vc, dtype), b.dt.expand(B, -1).contiguous(),
                             b.dl.expand(B).contiguous(), scale=1.0)
    got = oh.to_f32(host(got), dtype).astype(np.float64)
    for s in range(B):
        within(got[s * n:s * n + n], res, dtype, l, f"sequence {s}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 70], ids=["stream", "tiles"])
def test_roundings_of_one_sign(w4, n, dtype):
    """Nearly all probabilities round down, and those of the only keys with values up: the denominator is not rounded with them."""
    h, l = HALF[dtype], 192                  # (three blocks of 64: the tile's keys are not cut into pieces)
    scores = np.full(l, np.log1p(h * 0.98))  # 1 + 0.98 h: to 1
    scores[:64] = 0.0                        # the reference is taken from these
    up = 64 + 15 * np.arange(4)
    scores[up] = np.log1p(h * 1.02)          # to 1 + 2 h
    v = np.zeros((l, 64))
    v[up] = np.linspace(1.0, 2.0, 64)
    got, res = one_head(w4, n, scores, v, dtype)
    within(got, res, dtype, l, "one sign")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 70], ids=["stream", "tiles"])
def test_long_even_rows(w4, n, dtype):
    """30000 nearly equal scores, some powers of two above the first block's: the running sums take each block's as a whole."""
    rng = np.random.default_rng(21)
    l = 30000
    for above in (0.0, 3.9):
        scores = above + rng.uniform(-0.01, 0.01, l)
        scores[:64] = 0.0
        v = 1.0 + 0.1 * rng.standard_normal((l, 64))
        got, res = one_head(w4, n, scores, v, dtype)
        within(got, res, dtype, l, f"{above} above")


# (queries, keys) of every sequence; the second of each kind has rows at the border between the kernels
MIXED = [([(1, 20 + 9 * i) for i in range(100)] + [(256, 3000)], 8, 2, 64, 16), ([(32, 90)] * 30 + [(33, 60)] * 2 + [(400, 900), (3, 700)], 2, 2, 128, 16),
         ([(1, 300)] * 7 + [(17, 2000)] + [(1, 40)] * 7 + [(60, 900)], 1, 1, 128, 24), ([(4, 100)] * 40 + [(5, 90), (129, 2000), (2, 2)], 8, 1, 256, 32)]


@pytest.mark.parametrize("shape", MIXED, ids=[str(i) for i in range(len(MIXED))])
def test_short_sequences_among_long_ones(w4, shape):
    """The tiles of a batch of mostly short sequences, in both ways of numbering them: everything computed, within the workspace."""
    import torch
    print(f"\n{shape[1:]}", flush=True)
    b = Batch(30, *shape, "bf16", tail=7)
    for order in (False, True):
        if order:
            b = Batch(31, shape[0][::-1], *shape[1:], "bf16", tail=200)
        for max_q in (b.max_q, None):
            need = w4.attention_workspace_bytes(b.dq, b.dk, b.dv, len(b.both), max_q)
            ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
            out = torch.full_like(b.dq, 7.0)
            b.check(b.run(w4, workspace=ws[:need], out=out, max_q=max_q))
            assert (ws[need:] == 0xFF).all() and (out[int(b.starts[-1]):] == 7).all()
            m, pos = b.tree()
            b.check(b.run_tree(w4, m, pos, max_q=max_q), "tree", mask=m)


@pytest.mark.parametrize("each", [1, 9, 40])
def test_uniform_batch_with_a_loose_max_q(w4, each):
    """From C, a uniform batch (no q_starts) may state any max_q."""
    import ctypes
    import torch
    from w4a4_bit_quantized_amd import binding
    lib = w4.load_library()
    b = Batch(32, [(each, each + 11 * i) for i in range(50)], 4, 1, 64, 16, "bf16")
    cache, _ = binding._kv_cache(b.dk, b.dv, b.dq.dtype, b.dq.device)
    for max_q in (each, b.T, 1):
        out = torch.empty_like(b.dq)
        a = binding.Attention(b.dq.data_ptr(), 256, 64, out.data_ptr(), 256, 64, b.T, 4, b.dt.data_ptr(), b.dt.stride(0), b.dt.shape[1],
                              b.dl.data_ptr(), None, 50, max_q, 0, 0, 0.125, 64, 0)
        ra, rc = ctypes.byref(a), ctypes.byref(cache)
        ws = torch.empty(lib.w4a4_attention_workspace_bytes(ra, rc), dtype=torch.uint8, device="cuda")
        st = torch.cuda.current_stream().cuda_stream
        assert lib.w4a4_paged_attention(ra, rc, ws.data_ptr(), ws.numel(), st) == 0
        b.check(out, f"max_q = {max_q}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("strong", [2, 229], ids=["before", "after"])
@pytest.mark.parametrize("at", [40, 100, 240], ids=str)
@pytest.mark.parametrize("n", [1, 70], ids=["stream", "tiles"])
def test_infinite_values_of_no_weight(w4, n, at, strong, dtype):
    """An infinite value whose probability is 0 in float32, in blocks that a mask cuts and others, before and behind the largest
    score: that element of the rows that see it is infinite or NaN, everything else is as without it."""
    l, D = 300, 64
    b = Batch(33, [(n, l)], 1, 1, D, 16, dtype)
    k = oh.to_f32(b.kc, dtype)
    k[..., 0] = 0.0
    k[b.table[0, strong // 16], strong % 16, 0, 0] = 120.0
    q = oh.to_f32(b.q, dtype) * 0.05
    q[..., 0] = 1.0
    b.q, b.kc = oh.from_f32(q, dtype), oh.from_f32(k, dtype)
    b.dq, b.dk = dev(b.q, dtype), dev(b.kc, dtype)
    for window in (0, 220):  # (the first blocks of 64 are cut by the window, the last ones by the queries)
        kw = dict(window=window, sinks=3 if window else 0, scale=1.0)
        ref = oh.to_f32(host(b.run(w4, **kw)), dtype)
        b.check(b.run(w4, **kw), "without", **kw)
        old = b.dv.clone()
        b.dv[int(b.table[0, at // 16]), at % 16, 0, 5] = float("inf")
        got = oh.to_f32(host(b.run(w4, **kw)), dtype)
        b.dv = old
        p = l - n + np.arange(n)
        sees = (at <= p) & ((window == 0) | (at > p - window))
        assert not np.isfinite(got[sees, 0, 5]).any() and not (got[sees, 0, 5] == -np.inf).any()
        got[sees, 0, 5] = ref[sees, 0, 5]
        assert (got == ref).all()
