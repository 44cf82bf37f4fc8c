"""GPU parity of attention over the paged cache (needs an MI355X) against ``oracle/attention.py`` in 64 bits.

Tolerance of an output o = sum_j P_j v_j, with A = sum_j P_j |v_j| and h half a step of the type: a probability is off by
  h                                               its rounding for the second product,
  (D + 4) 2^-23 X                                 its score: D products, exact in float32, summed in float32 (each addition
                                                  rounded or cut off), scaled, and the largest taken off, where X is the
                                                  largest scale sum_d |q_d k_d| of the row,
  2^-21 (1 + B) and 2^-23 X (1 + B)               exp2 and the factors that rescale sums, one per block of 32 keys, of B,
                                                  each with a difference of two maxima of at most X / ln 2
of itself; the sums add 2^-23 B and 32 2^-23 in a block.  The denominator is off by the same without h, so that
|error| <= A (h + 2 e), and then the output's own half step.  In f16 a probability below 2^-14 is off by 2^-25 of the
largest: 2^-25 sum_j |v_j| / sum_j exp(score_j - largest).
"""

import numpy as np
import pytest

from oracle import attention as oa
from oracle import hadamard as oh
from test_gpu_w8a8 import dev, host

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25}


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import w4a4_bit_quantized_amd as w
    w.load_library()
    return w


def limit(res, dtype, D, keys):
    o, absolute, spread, small = res
    blocks = keys / 32 + 1
    e = (D + 4) * 2.0 ** -23 * spread + (2.0 ** -21 + 2.0 ** -23 * spread) * (1 + blocks) + 2.0 ** -23 * (blocks + 32)
    err = absolute * (HALF[dtype] + 2 * e[..., None])
    if dtype == "f16":
        err = err + 2.0 ** -25 * small
    return err + (np.abs(o) + err) * HALF[dtype] + TINY[dtype]


class Batch:
    """A batch of sequences with (queries, keys) each, their keys on shuffled pages of a pool whose other places hold
    ``poison`` (what nobody sees must not count)."""

    def __init__(self, seed, both, hq, hk, D, page, dtype, poison=np.nan, heads_first=False, tail=0, scale=1.0, spare=3):
        import torch
        rng = np.random.default_rng(seed)
        self.rng, self.both, self.dtype, self.hq, self.hk, self.D, self.page = rng, both, dtype, hq, hk, D, page
        need = [-(-l // page) for _, l in both]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(both), max(max(need), 1)), -1, np.int32)
        kc = np.full((self.pages, page, hk, D), poison, np.float32)
        vc = kc.copy()
        at = 0
        for b, (n, l) in enumerate(both):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            j = np.arange(l)
            kc[self.table[b, j // page], j % page] = rng.standard_normal((l, hk, D)) * scale
            vc[self.table[b, j // page], j % page] = rng.standard_normal((l, hk, D))
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in both])]).astype(np.int32)
        self.T = int(self.starts[-1]) + tail
        self.q = oh.from_f32((rng.standard_normal((self.T, hq, D)) * 1.5).astype(np.float32), dtype)
        self.kc, self.vc = oh.from_f32(kc, dtype), oh.from_f32(vc, dtype)
        self.lens = np.array([l for _, l in both], np.int32)
        self.max_q = max(n for n, _ in both)
        self.heads_first = heads_first
        self.dq, self.dk, self.dv = dev(self.q, dtype), dev(self.kc, dtype), dev(self.vc, dtype)
        if heads_first:
            self.dk, self.dv = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (self.dk, self.dv))
        i = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
        self.dt, self.dl, self.ds = i(self.table), i(self.lens), i(self.starts)

    def expected(self, **kw):
        f = lambda x: oh.to_f32(x, self.dtype)
        return oa.paged(f(self.q), f(self.kc), f(self.vc), self.table, self.lens, self.starts, kw.pop("scale", self.D ** -0.5), **kw)

    def check(self, got, what="", **kw):
        res = self.expected(**kw)
        o = res[0]
        g = oh.to_f32(host(got), self.dtype).astype(np.float64)
        rows = slice(0, int(self.starts[-1]))
        off = ~(np.abs(g - o) <= limit(res, self.dtype, self.D, self.lens.max()))[rows]
        at = np.argwhere(off)
        assert at.size == 0, (f"{what}: {len(at)} of {off.size} off, first {at[:3].tolist()}: {g[tuple(at[0])]} for {o[tuple(at[0])]}, "
                              f"rows {sorted(set(at[:, 0].tolist()))[:20]}")

    def run(self, w4, **kw):
        return w4.paged_attention(self.dq, self.dk, self.dv, self.dt, self.dl, q_starts=self.ds,
                                  **{"max_q": self.max_q, **kw})

    def tree(self, mask=None, positions=True):
        """Random trees over every sequence's queries, and its nodes' positions."""
        m = np.zeros((self.T, self.max_q), bool)
        pos = np.zeros(self.T, np.int32)
        for b, (n, l) in enumerate(self.both):
            for i in range(n):
                r = self.starts[b] + i
                pos[r] = l - n
                if i and self.rng.random() < 0.9:
                    up = r - self.rng.integers(1, min(i, 4) + 1)
                    m[r], pos[r] = m[up], pos[up] + 1
                m[r, i] = True
        return m, pos

    def run_tree(self, w4, mask, pos, **kw):
        import torch
        return w4.tree_attention(self.dq, self.dk, self.dv, self.dt, self.dl, torch.from_numpy(mask).cuda(), q_starts=self.ds,
                                 positions=torch.from_numpy(pos).cuda(), **{"max_q": self.max_q, **kw})


DTYPES = ["bf16", "f16"]
# (queries, keys) of every sequence; query heads, key / value heads, head size; page size
DECODE = [([(1, 1)], 1, 1, 64, 16), ([(1, 33), (1, 0), (1, 1000), (1, 64)], 8, 2, 128, 16), ([(1, 700)] * 3, 4, 4, 8, 1),
          ([(1, 300), (1, 5), (1, 129)], 14, 2, 80, 24), ([(1, 257), (1, 256)], 6, 1, 256, 50), ([(1, 4000)], 32, 8, 128, 16),
          ([(1, 90 + 7 * i) for i in range(70)], 4, 1, 72, 64), ([(1, 513)], 64, 1, 96, 256), ([(1, 2222)], 7, 7, 120, 3)]


def names(shape):
    return f"{len(shape[0])}seq-{shape[1]}h{shape[2]}-{shape[3]}-p{shape[4]}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", DECODE, ids=names)
def test_decode(w4, shape, dtype):
    both, hq, hk, D, page = shape
    print(f"\n{shape} {dtype}", flush=True)
    b = Batch(1, both, hq, hk, D, page, dtype, heads_first=hq == 8)
    b.check(b.run(w4))
    b.check(b.run(w4, window=100, sinks=4), "window", window=100, sinks=4)
    if page == 16:
        b.check(b.run(w4, window=1), "window of one", window=1)
        b.check(b.run(w4, window=130, sinks=70, scale=0.3), "many sinks", window=130, sinks=70, scale=0.3)


FEW = [([(3, 3), (5, 70), (0, 9), (1, 1), (4, 2)], 8, 2, 128, 16), ([(16, 500), (7, 31)], 4, 4, 64, 24),
       ([(8, 1000), (12, 40)], 8, 2, 256, 32), ([(64, 64)], 1, 1, 40, 16), ([(9, 300), (2, 2)], 14, 2, 80, 5)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", FEW, ids=names)
def test_few_queries_and_trees(w4, shape, dtype):
    both, hq, hk, D, page = shape
    print(f"\n{shape} {dtype}", flush=True)
    b = Batch(2, both, hq, hk, D, page, dtype, tail=2)
    b.check(b.run(w4), "causal")
    b.check(b.run(w4, window=20, sinks=3), "window", window=20, sinks=3)
    m, pos = b.tree()
    b.check(b.run_tree(w4, m, pos), "tree", mask=m)
    b.check(b.run_tree(w4, m, pos, window=33, sinks=2), "tree, window", mask=m, positions=pos, window=33, sinks=2)
    m[::3] = False  # rows that see no drafted token
    b.check(b.run_tree(w4, m, pos), "tree with empty rows", mask=m)


MANY = [([(70, 70)], 4, 1, 64, 16), ([(200, 200), (3, 50), (129, 300)], 2, 2, 128, 16), ([(40, 700), (90, 95)], 8, 1, 80, 24),
        ([(1, 400), (150, 150), (0, 7), (2, 2)], 4, 2, 256, 32), ([(65, 30)], 3, 3, 8, 1), ([(300, 1000)], 2, 1, 128, 256)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", MANY, ids=names)
def test_prompts_and_large_trees(w4, shape, dtype):
    both, hq, hk, D, page = shape
    print(f"\n{shape} {dtype}", flush=True)
    b = Batch(3, both, hq, hk, D, page, dtype, tail=3, heads_first=hq == 2)
    b.check(b.run(w4), "causal")
    b.check(b.run(w4, window=60, sinks=5), "window", window=60, sinks=5)
    b.check(b.run(w4, max_q=1), "another kernel")
    m, pos = b.tree()
    b.check(b.run_tree(w4, m, pos), "tree", mask=m)
    m[::5] = False
    b.check(b.run_tree(w4, m, pos, window=75, sinks=70), "tree, window", mask=m, positions=pos, window=75, sinks=70)


@pytest.mark.parametrize("shape", [([(500, 600), (512, 900)], 16, 2, 128, 128), ([(1, 5000)], 8, 1, 128, 16), ([(9, 700), (3, 80)], 8, 2, 64, 16),
                                   ([(100, 150), (1, 900), (0, 3)], 4, 1, 256, 16)], ids=names)
def test_workspace_of_exactly_its_size(w4, shape):
    """Nothing is written behind the workspace, or behind the output's last sequence; what they held before does not matter."""
    import torch
    b = Batch(4, *shape, "bf16", tail=5)
    for kw in (dict(), dict(max_q=None)):
        need = w4.attention_workspace_bytes(b.dq, b.dk, b.dv, len(b.both), kw.get("max_q", b.max_q))
        ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        out = torch.full_like(b.dq, 7.0)
        b.check(b.run(w4, workspace=ws[:need], out=out, **kw))
        assert (ws[need:] == 0xFF).all() and (out[int(b.starts[-1]):] == 7).all()
        with pytest.raises(ValueError, match="workspace holds"):
            b.run(w4, workspace=ws[:need - 1], **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf], ids=str)
@pytest.mark.parametrize("shape", [([(5, 100), (4, 4)], 4, 2, 64, 16), ([(20, 200)], 2, 1, 128, 16), ([(40, 40)], 4, 1, 128, 24), ([(9, 130)], 8, 1, 256, 16),
                                   ([(200, 260)], 2, 2, 64, 16), ([(150, 150)], 1, 1, 80, 32)], ids=names)
def test_values_that_some_rows_see(w4, shape, bad, dtype):
    """An infinity or NaN among the values or keys of one position reaches the rows that see it and no other."""
    import torch
    both, hq, hk, D, page = shape
    b = Batch(5, both, hq, hk, D, page, dtype)
    n, l = both[0]
    at = l - n + n // 2                                  # a position that the later half of the queries sees
    b.vc[b.table[0, at // page], at % page, 0, 3] = oh.from_f32(np.array([bad], np.float32), dtype)[0]
    b.vc[b.table[0, at // page], at % page, 0, D - 1] = oh.from_f32(np.array([-bad], np.float32), dtype)[0]
    b.dv = dev(b.vc, dtype)
    window = n // 3 + 1
    m, pos = b.tree()
    m[: n] = np.tril(np.ones((n, b.max_q), bool))        # every second node sees its chain, the others only themselves
    m[1:n:2] = np.eye(n, b.max_q, dtype=bool)[1::2]
    for what, got, kw in (("causal", b.run(w4), {}), ("window", b.run(w4, window=window), dict(window=window)),
                          ("tree", b.run_tree(w4, m, pos), dict(mask=m))):
        with np.errstate(invalid="ignore"):
            res = b.expected(**kw)
        g, o = oh.to_f32(host(got), dtype).astype(np.float64), res[0]
        assert (np.isfinite(g) == np.isfinite(o)).all(), what
        assert (np.isnan(g) == np.isnan(o)).all() and (g[np.isinf(g)] == o[np.isinf(o)]).all(), what
        fine = np.isfinite(o)
        with np.errstate(invalid="ignore"):
            assert (np.abs(g - o)[fine] <= limit(res, dtype, D, l)[fine]).all(), what
    b.kc[b.table[0, at // page], at % page, 0, 1] = oh.from_f32(np.array([np.nan], np.float32), dtype)[0]
    b.dk = dev(b.kc, dtype)
    g = oh.to_f32(host(b.run(w4)), dtype)
    group = hq // hk
    assert np.isfinite(g[:n // 2]).all() and np.isnan(g[n // 2:n, :group]).all()
    assert np.isfinite(g[n:]).all() and (hk == 1 or np.isfinite(g[:n, group:]).all())
