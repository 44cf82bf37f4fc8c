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


def test_strided_tensors(w4):
    """Queries from a fused projection's output, an output in a wider matrix, uniform batches in four dimensions, one key / value
    tensor of the pool, heads outside the tokens; only the addressed elements are written."""
    import torch
    b = Batch(6, [(3, 60), (3, 45)], 4, 2, 64, 16, "bf16")
    ref = b.run(w4)
    b.check(ref)
    qkv = torch.randn(b.T, 8 * 64 + 8, device="cuda").bfloat16()
    qkv[:, 64:64 + 256] = b.dq.view(b.T, -1)
    q = qkv[:, 64:64 + 256].view(b.T, 4, 64)
    wide = torch.full((b.T, 4 * 72 + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 16:].view(b.T, 4, 72)[..., :64]
    both = torch.stack([b.dk, b.dv], 1)                   # (pages, 2, page, heads, D)
    args = (both[:, 0], both[:, 1], b.dt, b.dl)
    assert w4.paged_attention(q, *args, q_starts=b.ds, out=out) is out
    assert torch.equal(out, ref) and (wide[:, :16] == 3).all() and (wide[:, 16:].view(b.T, 4, 72)[..., 64:] == 3).all()
    four = w4.paged_attention(b.dq.view(2, 3, 4, 64), *args)
    assert four.shape == (2, 3, 4, 64) and torch.equal(four.view_as(ref), ref)
    heads = torch.empty(4, b.T, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    w4.paged_attention(b.dq.transpose(0, 1).contiguous().transpose(0, 1), *args, max_q=3, q_starts=b.ds, out=heads)
    assert torch.equal(heads, ref)
    pools = [x.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3) for x in (b.dk, b.dv)]
    assert torch.equal(b.run(w4), w4.paged_attention(b.dq, *pools, b.dt, b.dl, q_starts=b.ds, max_q=3))


@pytest.mark.parametrize("n", [1, 40])
def test_bad_pages_and_lengths(w4, n):
    """Entries that name no page hold no keys, lengths are cut to the table's; sequences share pages; pages that no window
    reaches may hold anything."""
    import torch
    D, page = 128, 16
    b = Batch(7, [(n, 200), (n, 150), (n, 90)], 4, 2, D, page, "bf16")
    for entry, value in (((0, 3), -1), ((0, 7), b.pages), ((1, 0), 2 ** 31 - 1), ((2, 5), -2 ** 31)):
        b.table[entry] = value
    b.dt = torch.from_numpy(b.table).cuda()
    b.check(b.run(w4), "bad pages")
    b.check(b.run(w4, window=70, sinks=20), "bad pages, window", window=70, sinks=20)
    b = Batch(8, [(n, 200), (n, 150), (n, 90)], 4, 2, D, page, "f16")
    b.table[1, :9] = b.table[0, :9]                       # a shared prefix
    b.table[2, 1] = b.table[2, 0]                         # one page twice
    b.dt = torch.from_numpy(b.table).cuda()
    b.check(b.run(w4), "shared pages")
    b.lens[:] = [13 * page + 50, -5, 90]                  # the table has 13 pages a row
    b.dl = torch.from_numpy(b.lens).cuda()
    b.table[0, 12] = b.table[0, 0]
    b.dt = torch.from_numpy(b.table).cuda()
    b.check(b.run(w4), "lengths")
    lost = n + 30                                         # what the window has left before the first query
    b = Batch(9, [(n, 200)], 4, 2, D, page, "bf16")
    b.table[0, 1:(200 - lost - 16) // page] = -1
    b.dt = torch.from_numpy(b.table).cuda()
    b.check(b.run(w4, window=30, sinks=7), "pages given away", window=30, sinks=7)


def test_masks_that_say_the_same(w4):
    """A chain is the causal mask, a window of all keys none: the same bits."""
    import torch
    for both, hq, hk in (([(5, 60), (8, 8)], 4, 2), ([(70, 90), (33, 200)], 4, 1)):
        b = Batch(10, both, hq, hk, 64, 16, "bf16")
        ref = b.run(w4)
        m = np.tril(np.ones((b.max_q, b.max_q), bool))
        m = np.concatenate([m[:n] for n, _ in both])
        assert torch.equal(b.run_tree(w4, m, np.zeros(b.T, np.int32)), ref)
        wide = np.concatenate([m, np.zeros((b.T, 5), bool)], 1).astype(np.uint8) * 7
        assert torch.equal(b.run_tree(w4, wide[:, :-2], np.zeros(b.T, np.int32)), ref)
        assert torch.equal(b.run(w4, window=300), ref) and torch.equal(b.run(w4, window=2 ** 40, sinks=2 ** 40), ref)
        assert torch.equal(b.run(w4, sinks=3), ref)
        narrow = b.run_tree(w4, m[:, :3], np.zeros(b.T, np.int32))  # columns past the mask are not seen
        b.check(narrow, "narrow mask", mask=m[:, :3])


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_scores(w4, dtype):
    """Peaked rows: scores of hundreds, whose running maximum rises from block to block."""
    for both in ([(1, 700), (2, 90)], [(80, 700)]):
        b = Batch(11, both, 4, 1, 128, 16, dtype, scale=4.0)
        b.check(b.run(w4, scale=1.0), "peaked", scale=1.0)
        b.check(b.run(w4, scale=1e-4), "flat", scale=1e-4)


def test_mixed_batch(w4):
    """One prompt among single tokens: two kernels share the launch's workspace."""
    for dtype in DTYPES:
        b = Batch(12, [(1, 50), (90, 300), (1, 400), (2, 3), (1, 1)] + [(1, 20 + i) for i in range(40)], 8, 2, 64, 16, dtype)
        b.check(b.run(w4), "mixed")
        m, pos = b.tree()
        b.check(b.run_tree(w4, m, pos, window=30, sinks=2), "mixed trees", mask=m, positions=pos, window=30, sinks=2)


def test_many_sequences(w4):
    """More sequences than lanes, most of them empty or short, some without queries."""
    rng = np.random.default_rng(13)
    both = [(int(n), int(n + l)) for n, l in zip(rng.integers(0, 3, 300), rng.integers(0, 60, 300) * rng.integers(0, 2, 300))]
    b = Batch(13, both, 2, 1, 64, 16, "bf16")
    b.check(b.run(w4))
    b.check(b.run(w4, window=9, sinks=1, max_q=b.T), "tiles", window=9, sinks=1)


def test_far_offsets(w4):
    """Pages whose elements lie more than 2^32 elements into the pool give what near ones give."""
    import torch
    D, page, hk = 128, 16, 2
    for n in (1, 60):
        b = Batch(14, [(n, 150), (n, 99)], 4, hk, D, page, "bf16")
        ref = b.run(w4)
        pages = (1 << 32) // (page * hk * D) + b.pages + 5
        pool = torch.empty(pages, page, hk, 2 * D, dtype=torch.bfloat16, device="cuda")  # 17 GB
        k, v = pool[..., :D], pool[..., D:]
        k[-b.pages:], v[-b.pages:] = b.dk, b.dv
        far = torch.where(b.dt >= 0, b.dt + (pages - b.pages), b.dt)
        assert torch.equal(w4.paged_attention(b.dq, k, v, far, b.dl, q_starts=b.ds, max_q=n), ref)
        slots = torch.tensor([(pages - 1) * page + 3], device="cuda")
        new = torch.randn(1, hk, D, device="cuda").bfloat16()
        w4.kv_append(None, new, new + 1, None, [], slots, k, v, norm=False)
        assert torch.equal(k[-1, 3], new[0]) and torch.equal(v[-1, 3], (new + 1)[0])
        del pool, k, v


def test_streams_and_graphs(w4):
    """Calls on two streams at once; a captured step of append and attention, replayed on new data with eager work between;
    two graphs that share a workspace; every replay gives the eager bits."""
    import torch
    D, page, hq, hk, B = 64, 16, 8, 2, 6
    b = Batch(15, [(1, 30 + 40 * i) for i in range(B)], hq, hk, D, page, "bf16", poison=0.0)
    c = Batch(16, [(50, 120), (60, 300)], hq, hk, D, page, "bf16", poison=0.0)
    refs = [b.run(w4), c.run(w4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        outs = []
        for st, x in zip(streams, (b, c)):
            with torch.cuda.stream(st):
                outs.append(x.run(w4))
        torch.cuda.synchronize()
        assert torch.equal(outs[0], refs[0]) and torch.equal(outs[1], refs[1])

    ws = torch.empty(max(w4.attention_workspace_bytes(x.dq, x.dk, x.dv, len(x.both), x.max_q) for x in (b, c)), dtype=torch.uint8,
                     device="cuda")
    q, kv = torch.randn(B, hq, D, device="cuda").bfloat16(), torch.randn(2, B, hk, D, device="cuda").bfloat16()
    lens, slots, pos = b.dl.clone(), torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    out, qo, oc = torch.empty_like(q), torch.empty_like(q), torch.empty_like(c.dq)
    dk, dv = b.dk.clone(), b.dv.clone()

    def step():
        w4.kv_append(q, kv[0], kv[1], pos, [D], slots, dk, dv, layout="half", q_out=qo)
        w4.paged_attention(qo, dk, dv, b.dt, lens, workspace=ws, out=out)

    step()
    c.run(w4, workspace=ws, out=oc)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        step()
    with torch.cuda.graph(graphs[1]):
        c.run(w4, workspace=ws, out=oc)
    for i in range(6):
        q.copy_(torch.randn_like(q))
        kv.copy_(torch.randn_like(kv))
        lens.copy_(torch.clamp(b.dl - i * 3, min=1))
        pos.copy_(lens - 1)
        last = (lens - 1).long()
        slots.copy_(b.dt[torch.arange(B, device="cuda"), last // page].long() * page + last % page)
        saved = dk.clone(), dv.clone()
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        got, kept = out.clone(), (dk.clone(), dv.clone())
        dk.copy_(saved[0])
        dv.copy_(saved[1])
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(kept[0], dk) and torch.equal(kept[1], dv) and torch.equal(oc, refs[1])


def test_serving_steps(w4):
    """A prompt in two pieces, decoded tokens, then drafted ones, through projection, append, attention and projection, each step
    against attention over everything appended so far."""
    import torch
    rng = np.random.default_rng(17)
    D, hq, hk, page, width = 64, 4, 2, 16, 256
    K = hq * D
    lin = lambda n, k: dict(zip(("qweight", "wscales"), w4.w8a8_quantize_weight(torch.randn(n, k, device="cuda").bfloat16() / k ** 0.5)))
    qkv_l, out_l = lin((hq + 2 * hk) * D, width), lin(width, K)
    pool = [torch.full((30, page, hk, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.from_numpy(rng.permutation(30).astype(np.int32)).cuda().view(2, 15)
    done = [0, 0]
    f = lambda t: t.float().cpu().numpy().astype(np.float64)
    for ns, mask in (((40, 17), None), ((25, 60), None), ((1, 1), None), ((1, 1), None), ((6, 6), np.array(
            [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 0, 1, 0, 0, 0], [1, 1, 0, 1, 0, 0], [1, 0, 1, 0, 1, 0], [1, 1, 0, 1, 0, 1]], bool))):
        T = sum(ns)
        x = torch.randn(T, width, device="cuda").bfloat16()
        q, k, v = (t.view(T, -1, D) for t in w4.w8a8_linear(x, qkv_l).split([hq * D, hk * D, hk * D], 1))
        at = torch.cat([torch.arange(done[s], done[s] + n, device="cuda") for s, n in enumerate(ns)])
        which = torch.repeat_interleave(torch.arange(2, device="cuda"), torch.tensor(ns, device="cuda"))
        depth = at if mask is None else torch.tensor([done[s] + int(r.sum()) - 1 for s in range(2) for r in mask], device="cuda")
        slots = table[which, at // page].long() * page + at % page
        q = w4.kv_append(q, k, v, depth, [D], slots, *pool, layout="half")
        done = [d + n for d, n in zip(done, ns)]
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, ns[0], T], dtype=torch.int32, device="cuda")
        kw = dict(q_starts=starts, max_q=max(ns), window=48, sinks=4)
        m = None if mask is None else np.concatenate([mask, mask])
        if mask is None:
            o = w4.paged_attention(q, *pool, table, lens, **kw)
        else:
            o = w4.tree_attention(q, *pool, table, lens, torch.from_numpy(m).cuda(), positions=depth.int(), **kw)
        y = w4.w8a8_linear(o.view(T, K), out_l)
        res = oa.paged(f(q), f(pool[0]), f(pool[1]), table.cpu().numpy(), done, [0, ns[0], T], D ** -0.5, window=48, sinks=4, mask=m,
                       positions=depth.cpu().numpy())
        assert (np.abs(f(o) - res[0]) <= limit(res, "bf16", D, max(done))).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("n", [3, 40])
def test_mask_of_no_columns(w4, n):
    """No drafted token sees another: only the keys before the tree, none of a sequence that has none; numbers past 64 bits."""
    import torch
    b = Batch(19, [(n, 150), (n, n), (n - 1, 70)], 4, 2, 64, 16, "bf16")
    m = np.zeros((b.T, 0), np.uint8)
    b.check(b.run_tree(w4, m, np.zeros(b.T, np.int32)), "no columns", mask=m)
    assert torch.equal(b.run(w4, max_q=2 ** 80), b.run(w4, max_q=b.T))
    for bad in (dict(window=2 ** 64 + 5), dict(window=9, sinks=2 ** 63)):
        with pytest.raises(ValueError, match="out of range"):
            b.run(w4, **bad)


def test_refusals(w4):
    import torch
    b = Batch(18, [(1, 20), (2, 9)], 4, 2, 64, 16, "bf16")
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    args = dict(k_cache=b.dk, v_cache=b.dv, page_table=b.dt, kv_lens=b.dl, q_starts=b.ds)
    for bad, err in ((dict(k_cache=b.dk.half()), TypeError), (dict(k_cache=b.dk[..., :32]), ValueError), (dict(v_cache=b.dv[:1]), ValueError),
                     (dict(page_table=b.dt.long()), TypeError), (dict(page_table=b.dt[0]), ValueError), (dict(kv_lens=b.dl[:1]), ValueError),
                     (dict(q_starts=b.ds[:2]), ValueError), (dict(q_starts=b.ds.long()), TypeError), (dict(kv_lens=b.dl.cpu()), ValueError),
                     (dict(q_starts=None), ValueError), (dict(max_q=-1), ValueError), (dict(window=-1), w4.W4A4Error),
                     (dict(scale=0.0), w4.W4A4Error), (dict(out=z(3, 4, 32)), ValueError), (dict(out=b.dq), w4.W4A4Error),
                     (dict(workspace=z(10, dtype=torch.uint8)), ValueError), (dict(page_table=b.dt.t()), ValueError)):
        with pytest.raises(err):
            w4.paged_attention(b.dq, **{**args, **bad})
    with pytest.raises(ValueError, match="heads"):
        w4.paged_attention(z(3, 3, 64), **args)
    with pytest.raises(TypeError):
        w4.paged_attention(b.dq.float(), **args)
    with pytest.raises(w4.W4A4Error, match="ALIGN"):
        w4.paged_attention(z(3 * 4 * 64 + 1)[1:].view(3, 4, 64), **args)
    m = torch.ones(3, 2, dtype=torch.bool, device="cuda")
    for bad, err in ((dict(tree_mask=m[:2]), ValueError), (dict(tree_mask=m.int()), TypeError), (dict(window=3), ValueError),
                     (dict(window=3, positions=z(2, dtype=torch.int32)), ValueError), (dict(window=3, positions=z(3, dtype=torch.int64)), TypeError)):
        with pytest.raises(err):
            w4.tree_attention(b.dq, **{**args, "tree_mask": m, **bad})
    k = z(3, 2, 64)
    good = dict(q=None, k=k, v=k, positions=z(3, dtype=torch.int32), axis_dims=[64], slots=z(3, dtype=torch.int64), k_cache=b.dk, v_cache=b.dv)
    for bad, err in ((dict(slots=z(2, dtype=torch.int64)), ValueError), (dict(slots=z(3)), TypeError), (dict(v=z(3, 1, 64)), ValueError),
                     (dict(k=z(3, 2, 32)), ValueError), (dict(k=k.float()), TypeError), (dict(q_out=k), ValueError), (dict(inplace=True), ValueError),
                     (dict(v_cache=b.dk), w4.W4A4Error), (dict(layout="other"), ValueError), (dict(positions=z(4, dtype=torch.int32)), ValueError),
                     (dict(k_cache=b.dk[:, :1].expand(-1, 16, -1, -1)), w4.W4A4Error)):
        with pytest.raises(err):
            w4.kv_append(**{**good, **bad})
