"""GPU parity of the q / k head norm with rotary positions (needs an MI355X) against
``oracle/rope.py`` in 64 bits.

Tolerance, per element of a rotated pair (u0, u1) with s = |u0| + |u1|, in units of 2^-24 of s: the sum
of squares collects 8 products in a lane and at most 6 exchange steps (14 roundings, halved by the
square root: 7), the mean and eps 2 (halved: 1), rsqrt 4 (two units in the last place), x * r and
* weight 2, sincospi 4 (two units in the last place) and its rounded argument pi / 2 (the angle is
rounded to 2^-25 half turns of at most 1, that is pi 2^-25 in the sine), the rotation 2: below 22.
The angle in float64 adds |angle| * 6 * 2^-53.  Then half a unit in the last place of the storage type.
"""

import numpy as np
import pytest

from oracle import hadamard as oh
from oracle import rope as orope
from test_gpu_w8a8 import DTYPES, dev, host, tdtype

pytestmark = pytest.mark.gpu

HALF_ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}  # a subnormal's step


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import w4a4_bit_quantized_amd as w
    w.load_library()
    return w


def bound(u, y, dtype, dims, layout, shared, theta, pos):
    s = np.abs(u)
    far = np.zeros(u.shape[0])
    for e0, e1, a, ex in orope.pair_table(dims, layout, shared):
        s[..., e0] = s[..., e1] = np.abs(u[..., e0]) + np.abs(u[..., e1])
        far = np.maximum(far, np.abs(pos[:, a].astype(np.float64)) * theta ** -ex)
    err = s * (22 * 2.0 ** -24 + far[:, None, None] * 6 * 2.0 ** -53)
    return err + (np.abs(y) + err) * HALF_ULP[dtype] + TINY[dtype]


def check(got, x, pos, dims, dtype, weight=None, layout="interleaved", shared=False, norm=True, theta=10000.0, eps=1e-6,
          what=""):
    y, u = orope.norm_rope(oh.to_f32(x, dtype), pos, dims, None if weight is None else oh.to_f32(weight, dtype), eps,
                           theta, layout, shared, norm)
    g = oh.to_f32(host(got), dtype).astype(np.float64)
    assert g.shape == y.shape
    lim = bound(u, y, dtype, dims, layout, shared, theta, np.asarray(pos).reshape(len(y), len(dims)))
    over = np.abs(g - y) > lim
    at = np.argwhere(over)
    assert at.size == 0, f"{what}: {len(at)} of {g.size} off, first {at[:3].tolist()}: {g[tuple(at[0])]} for {y[tuple(at[0])]}"


def make(rng, T, H, D, dtype, scale=1.5):
    return oh.from_f32((rng.standard_normal((T, H, D)) * scale).astype(np.float32), dtype)


def weights(rng, D, dtype):
    return oh.from_f32(rng.uniform(0.5, 1.5, D).astype(np.float32), dtype)


def run(w4, rng, T, hq, hk, D, dims, dtype, layout, shared=False, weight=True, norm=True, far=1000, pos64=False, **kw):
    import torch
    print(f"\nT={T} heads={hq}+{hk} D={D} axes={dims} {dtype} {layout}", flush=True)
    q, k = make(rng, T, hq, D, dtype), make(rng, T, hk, D, dtype)
    qw, kw_ = (weights(rng, D, dtype), weights(rng, D, dtype)) if weight else (None, None)
    pos = rng.integers(-far, far + 1, (T, len(dims)))
    pt = torch.from_numpy(pos.astype(np.int64 if pos64 else np.int32)).cuda()
    yq, yk = w4.qk_norm_rope(dev(q, dtype), dev(k, dtype), pt, dims, None if qw is None else dev(qw, dtype),
                             None if kw_ is None else dev(kw_, dtype), layout=layout, shared_frequencies=shared,
                             norm=norm, **kw)
    torch.cuda.synchronize()
    o = {n: kw[n] for n in ("theta", "eps") if n in kw}
    check(yq, q, pos, dims, dtype, qw, layout, shared, norm, what="q", **o)
    check(yk, k, pos, dims, dtype, kw_, layout, shared, norm, what="k", **o)


LAYOUTS = ["interleaved", "half", "axis_half"]
SHAPES = [(1, 1, 1, 64, [64]), (1, 32, 8, 128, [128]), (5, 3, 1, 128, [16, 56, 56]), (130, 24, 24, 128, [44, 42, 42]),
          (600, 4, 2, 80, [16, 24, 24]), (4100, 5, 3, 64, [8, 24, 32]), (33, 2, 2, 256, [64, 64, 64, 64]),
          (7, 3, 2, 512, [128, 256]), (9, 2, 1, 34, [2, 10, 6]), (3, 1, 1, 2, [2]), (17, 2, 3, 120, [40, 0, 48]),
          (4101, 3, 1, 6, [2, 2]), (2, 2, 1, 512, [510]), (70, 40, 2, 16, [8])]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(w4, shape, layout):
    """Head sizes, head counts, axes (an empty one among them), part of the head rotated; every type."""
    for i, dtype in enumerate(DTYPES):
        rng = np.random.default_rng(i + shape[0])
        run(w4, rng, *shape, dtype, layout, shared=i == 1, pos64=i == 2)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_without_norm_or_weight(w4, layout):
    rng = np.random.default_rng(3)
    run(w4, rng, 20, 6, 2, 128, [32, 48, 48], "bf16", layout, weight=False)
    run(w4, rng, 20, 6, 2, 128, [32, 48, 48], "f32", layout, norm=False)
    run(w4, rng, 20, 6, 2, 72, [30, 42], "f16", layout, norm=False, weight=False)


def test_far_positions_and_parameters(w4):
    """Positions up to the ends of their types lose no accuracy; other theta and eps."""
    rng = np.random.default_rng(4)
    run(w4, rng, 64, 2, 1, 64, [64], "f32", "half", far=2 ** 31 - 1)
    run(w4, rng, 64, 2, 1, 64, [32, 32], "f32", "interleaved", far=2 ** 40, pos64=True, shared=True)
    run(w4, rng, 64, 2, 1, 64, [64], "f32", "half", far=500000, theta=5e5, eps=1e-5)
    run(w4, rng, 64, 2, 1, 64, [64], "f32", "interleaved", far=1000, theta=0.5, eps=0.0)


def test_norm_only(w4):
    import torch
    rng = np.random.default_rng(5)
    for dtype in DTYPES:
        x, w = make(rng, 40, 3, 128, dtype), weights(rng, 128, dtype)
        y = w4.qk_norm_rope(dev(x, dtype), None, None, [], q_weight=dev(w, dtype))
        assert isinstance(y, torch.Tensor)
        check(y, x, np.zeros((40, 0)), [], dtype, w)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("start", [0, 3, 8])
def test_partitions_in_place(w4, dtype, start):
    """q and k partitions of a fused projection's rows, in place: v, the columns before them and the
    rows behind the last token stay as they were, and the result is the out-of-place one."""
    import torch
    rng = np.random.default_rng(start)
    T, hq, hk, D, dims = 50, 6, 2, 96, [24, 32, 40]
    width = start + (hq + 2 * hk) * D
    big = dev(oh.from_f32(rng.standard_normal((T + 3, width)).astype(np.float32), dtype), dtype)
    before = big.clone()
    q = big[:T, start:start + hq * D].unflatten(1, (hq, D))
    k = big[:T, start + hq * D:start + (hq + hk) * D].unflatten(1, (hk, D))
    qh, kh = host(q), host(k)
    pos = torch.from_numpy(rng.integers(0, 99, (T, 3)).astype(np.int32)).cuda()
    wq, wk = weights(rng, D, dtype), weights(rng, D, dtype)
    for layout in LAYOUTS:
        big.copy_(before)
        a, b = w4.qk_norm_rope(q, k, pos, dims, dev(wq, dtype), dev(wk, dtype), layout=layout)
        assert torch.equal(big, before)
        w4.qk_norm_rope(q, k, pos, dims, dev(wq, dtype), dev(wk, dtype), layout=layout, inplace=True)
        assert torch.equal(q, a) and torch.equal(k, b)
        keep = torch.ones_like(big, dtype=torch.bool)
        keep[:T, start:start + (hq + hk) * D] = False
        assert torch.equal(big[keep], before[keep])
        check(a, qh, pos.cpu().numpy(), dims, dtype, wq, layout)
        check(b, kh, pos.cpu().numpy(), dims, dtype, wk, layout)


def test_head_major_output_batches_and_broadcast(w4):
    """(heads, tokens, head_dim) outputs, 4-D inputs, a broadcast key head; one query head alone."""
    import torch
    rng = np.random.default_rng(8)
    B, S, hq, hk, D, dims = 3, 11, 4, 2, 64, [16, 48]
    q, k = make(rng, B * S, hq, D, "bf16"), make(rng, B * S, 1, D, "bf16")
    pos = rng.integers(0, 50, (B, S, 2)).astype(np.int32)
    qd = dev(q, "bf16").view(B, S, hq, D)
    kd = dev(k, "bf16").expand(B * S, hk, D)
    pt = torch.from_numpy(pos).cuda()
    q_out = torch.empty((hq, B * S, D), dtype=torch.bfloat16, device="cuda")
    a = w4.qk_norm_rope(qd.view(B * S, hq, D), None, pt.view(B * S, 2), dims, q_out=q_out.transpose(0, 1))
    b, kk = w4.qk_norm_rope(qd, kd, pt, dims)
    assert tuple(b.shape) == (B, S, hq, D) and tuple(kk.shape) == (B * S, hk, D)
    assert torch.equal(a, b.view(B * S, hq, D)) and torch.equal(q_out.transpose(0, 1), a)
    check(a, q, pos.reshape(-1, 2), dims, "bf16")
    check(kk, np.repeat(k, hk, 1), pos.reshape(-1, 2), dims, "bf16")


def test_special_values_stay_in_their_head(w4):
    """Zero heads stay zero; an infinity or a NaN reaches its own head only."""
    import torch
    rng = np.random.default_rng(9)
    q = dev(make(rng, 6, 3, 128, "f32"), "f32")
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    clean = w4.qk_norm_rope(q, None, pos, [128])
    q[1, 1] = 0.0
    q[2, 0, 5], q[4, 2, 100] = float("inf"), float("nan")
    y = w4.qk_norm_rope(q, None, pos, [128])
    assert bool((y[1, 1] == 0).all())
    assert bool(y[2, 0].isnan().any()) and bool(y[4, 2].isnan().all())
    for t, h in ((1, 1), (2, 0), (4, 2)):
        y[t, h] = clean[t, h]
    assert torch.equal(y, clean)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_elements_past_the_span_are_kept(w4, layout, dtype):
    """Without the norm, elements past the rotary span leave bit for bit, infinities, NaNs and signed zeros
    beside each other too; the rotated ones are not touched by them."""
    import torch
    rng = np.random.default_rng(11)
    special = np.array([np.inf, 1.0, -0.0, -1.0, np.nan, 2.0, 0.0, -np.inf, 3.0, 1e-8], np.float32)
    for D, dims in ((64, [8, 16]), (64, [6]), (66, [24, 8]), (128, [16, 2, 6]), (132, [2]), (16, [])):
        rot = sum(dims)
        xf = oh.to_f32(make(rng, 5, 3, D, dtype), dtype).copy()
        xf[..., rot:] = np.resize(special, (5, 3, D - rot))
        x = oh.from_f32(xf, dtype)
        pos = rng.integers(0, 50, (5, len(dims)))
        pt = torch.from_numpy(pos.astype(np.int32)).cuda() if dims else None
        got = host(w4.qk_norm_rope(dev(x, dtype), None, pt, dims, layout=layout, norm=False))
        past, want = got[..., rot:], np.ascontiguousarray(x[..., rot:])
        nan = np.isnan(oh.to_f32(want, dtype))
        assert (np.isnan(oh.to_f32(past, dtype)) == nan).all(), f"D={D} axes={dims}"
        assert (np.ascontiguousarray(past).view(np.uint8).reshape(*past.shape, -1)[~nan]
                == want.view(np.uint8).reshape(*want.shape, -1)[~nan]).all(), f"D={D} axes={dims}"
        if rot:
            zero = xf.copy()
            zero[..., rot:] = 0
            y = host(w4.qk_norm_rope(dev(oh.from_f32(zero, dtype), dtype), None, pt, dims, layout=layout, norm=False))
            assert (got[..., :rot] == y[..., :rot]).all()


def test_weights_that_do_not_count(w4):
    """Through the C interface: the weight of a tensor without heads is not read (here its address is not one of
    the type's), and without the norm no weight is applied."""
    import ctypes
    import torch
    from w4a4_bit_quantized_amd import binding
    lib = w4.load_library()
    x = torch.randn(5, 2, 64, device="cuda")
    w = torch.full((66,), 3.0, device="cuda")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    dims = (ctypes.c_int32 * 1)(64)
    for flags, weight in ((1, None), (0, w)):
        y = torch.zeros_like(x)
        none = binding.Heads(None, 0, 0, 0, w.data_ptr() + 1, None, 0, 0)
        some = binding.Heads(x.data_ptr(), 128, 64, 2, None if weight is None else w.data_ptr(), y.data_ptr(), 128, 64)
        st = lib.w4a4_qk_norm_rope(ctypes.byref(none), ctypes.byref(some), pos.data_ptr(), 5, 64, 1, dims, 0, flags,
                                   1e4, 1e-6, 2, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        want = w4.qk_norm_rope(x, None, pos, [64], norm=bool(flags))
        assert torch.equal(y, want)


def test_empty_and_refused_calls(w4):
    import torch
    q = torch.zeros((4, 2, 64), device="cuda")
    p = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    a, b = w4.qk_norm_rope(q[:0], q[:0, :1], p[:0], [64])
    assert a.shape[0] == 0 and b.shape[0] == 0
    assert w4.qk_norm_rope(q[:, :0], None, p, [64]).numel() == 0
    for bad, err in ((dict(axis_dims=[66]), "ERR_SHAPE"), (dict(axis_dims=[33]), "ERR_SHAPE"),
                     (dict(axis_dims=[-2]), "ERR_SHAPE"), (dict(theta=0.0), "ERR_SHAPE"), (dict(eps=-1.0), "ERR_SHAPE"),
                     (dict(theta=float("nan")), "ERR_SHAPE"),
                     (dict(q_out=torch.zeros((1, 1, 64), device="cuda").expand(4, 2, 64)), "ERR_SHAPE")):
        with pytest.raises(w4.W4A4Error, match=err):
            w4.qk_norm_rope(q, None, p, **{"axis_dims": [64], **bad})
    with pytest.raises(w4.W4A4Error, match="ERR_SHAPE"):
        w4.qk_norm_rope(q[..., :33], None, p, [32])
    with pytest.raises(w4.W4A4Error, match="ERR_UNSUPPORTED"):
        w4.qk_norm_rope(torch.zeros((2, 1, 514), device="cuda"), None, p[:2], [64])
    with pytest.raises(w4.W4A4Error, match="ERR_UNSUPPORTED"):
        w4.qk_norm_rope(q, None, torch.zeros((4, 9), dtype=torch.int32, device="cuda"), [2] * 9)
    for kw, exc in ((dict(layout="other"), ValueError), (dict(q_weight=torch.ones(32, device="cuda")), ValueError),
                    (dict(q_weight=torch.ones(64, device="cuda", dtype=torch.bfloat16)), TypeError),
                    (dict(q_out=torch.zeros((4, 2, 32), device="cuda")), ValueError), (dict(inplace=True, q_out=q), ValueError)):
        with pytest.raises(exc):
            w4.qk_norm_rope(q, None, p, [64], **kw)
    with pytest.raises(ValueError, match="positions"):
        w4.qk_norm_rope(q, None, p[:3], [64])
    with pytest.raises(TypeError, match="positions"):
        w4.qk_norm_rope(q, None, p.float(), [64])
    with pytest.raises(ValueError, match="k has"):
        w4.qk_norm_rope(q, q[:3], p, [64])
    with pytest.raises(ValueError, match="flatten"):
        w4.qk_norm_rope(torch.zeros((2, 8, 2, 64), device="cuda")[:, :2], None, p, [64])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,dims", [(128, [44, 42, 42]), (64, [20, 2]), (96, [32, 64]), (90, [30, 60])])
def test_every_alignment(w4, dtype, D, dims):
    """Heads, strides, weights and outputs at element offsets 0 .. 8, in place too; the elements around the heads
    stay as they were."""
    import torch
    rng = np.random.default_rng(D)
    T, hq, hk = 9, 3, 2
    q, k, wq, wk = make(rng, T, hq, D, dtype), make(rng, T, hk, D, dtype), weights(rng, D, dtype), weights(rng, D, dtype)
    pos = rng.integers(0, 500, (T, len(dims)))
    pt = torch.from_numpy(pos.astype(np.int32)).cuda()
    for off in range(9):
        pad = off % 3  # elements between the heads
        big = torch.full((T + 1, off + (hq + hk) * (D + pad) + 1), 5.0, dtype=tdtype(dtype), device="cuda")
        heads = big[:T, off:off + (hq + hk) * (D + pad)].unflatten(1, (hq + hk, D + pad))[..., :D]
        heads[:, :hq], heads[:, hq:] = dev(q, dtype), dev(k, dtype)
        w = torch.full((2 * D + 9,), 5.0, dtype=tdtype(dtype), device="cuda")
        w[off:off + D], w[off + D:off + 2 * D] = dev(wq, dtype), dev(wk, dtype)
        before = big.clone()
        outs = torch.zeros_like(big)
        to = outs[:T, off:off + (hq + hk) * (D + pad)].unflatten(1, (hq + hk, D + pad))[..., :D]
        for layout in LAYOUTS:
            big.copy_(before)
            a, b = w4.qk_norm_rope(heads[:, :hq], heads[:, hq:], pt, dims, w[off:off + D], w[off + D:off + 2 * D],
                                   layout=layout, q_out=to[:, :hq], k_out=to[:, hq:])
            assert torch.equal(big, before)
            check(a, q, pos, dims, dtype, wq, layout, what=f"q off {off}")
            check(b, k, pos, dims, dtype, wk, layout, what=f"k off {off}")
            w4.qk_norm_rope(heads[:, :hq], heads[:, hq:], pt, dims, w[off:off + D], w[off + D:off + 2 * D], layout=layout,
                            inplace=True)
            assert torch.equal(heads, to)
            heads.copy_(before[:T, off:off + (hq + hk) * (D + pad)].unflatten(1, (hq + hk, D + pad))[..., :D])
            assert torch.equal(big, before), "elements around the heads were written"
        to.zero_()
        assert not bool(outs.any()), "elements around the output heads were written"


def test_one_tensor_as_q_and_k(w4):
    """One input for both (with different weights), broadcast tokens and heads, on two streams at once."""
    import torch
    rng = np.random.default_rng(31)
    T, H, D, dims = 40, 6, 96, [32, 64]
    x, a, b = make(rng, T, H, D, "bf16"), weights(rng, D, "bf16"), weights(rng, D, "bf16")
    pos = rng.integers(0, 500, (T, 2))
    xt, pt = dev(x, "bf16"), torch.from_numpy(pos).cuda()
    row, head = dev(x[:1], "bf16").expand(T, H, D), dev(x[:, :1], "bf16").expand(T, H, D)
    torch.cuda.synchronize()
    got = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            got.append((w4.qk_norm_rope(xt, xt, pt, dims, dev(a, "bf16"), dev(b, "bf16"), layout="half"),
                        w4.qk_norm_rope(row, head, pt, dims, layout="axis_half")))
    torch.cuda.synchronize()
    for (q, k), (r, h) in got:
        check(q, x, pos, dims, "bf16", a, "half")
        check(k, x, pos, dims, "bf16", b, "half")
        check(r, np.repeat(x[:1], T, 0), pos, dims, "bf16", None, "axis_half")
        check(h, np.repeat(x[:, :1], H, 1), pos, dims, "bf16", None, "axis_half")
    with pytest.raises(w4.W4A4Error, match="ERR_SHAPE"):
        w4.qk_norm_rope(xt, xt, pt, dims, inplace=True)


def test_graph_replay(w4):
    import torch
    rng = np.random.default_rng(10)
    q, k = dev(make(rng, 90, 8, 128, "bf16"), "bf16"), dev(make(rng, 90, 2, 128, "bf16"), "bf16")
    pos = torch.zeros((90, 3), dtype=torch.int32, device="cuda")
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    args = (q, k, pos, [16, 56, 56])
    w4.qk_norm_rope(*args, q_out=oq, k_out=ok)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.qk_norm_rope(*args, q_out=oq, k_out=ok)
    for _ in range(4):
        q.copy_(dev(make(rng, 90, 8, 128, "bf16"), "bf16"))
        pos.copy_(torch.from_numpy(rng.integers(0, 100, (90, 3)).astype(np.int32)))
        a, b = w4.qk_norm_rope(*args)
        oq.zero_()
        ok.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(oq, a) and torch.equal(ok, b)


def test_projection_then_norm_and_rotation(w4):
    """As they are used together: one quantized activation, a fused 8-bit q / k / v projection into one
    matrix, q and k normed and rotated in place, then rotated per head by the block Hadamard transform;
    the same with the 4-bit layer's output."""
    import torch
    from oracle import w8a8 as ow
    rng = np.random.default_rng(12)
    T, K, hq, hk, D, dims = 77, 512, 4, 2, 64, [16, 24, 24]
    N = (hq + 2 * hk) * D
    x = oh.from_f32(rng.standard_normal((T, K)).astype(np.float32), "bf16")
    lam = oh.from_f32(rng.uniform(0.5, 2, K).astype(np.float32), "bf16")
    w = oh.from_f32((rng.standard_normal((N, K)) * K ** -0.5).astype(np.float32), "bf16")
    qw, sw = w4.w8a8_quantize_weight(dev(w, "bf16"), dev(lam, "bf16"), hadamard_block=64)
    qkv = w4.w8a8_linear(dev(x, "bf16"), dict(qweight=qw, wscales=sw, smooth_factor=dev(lam, "bf16")), hadamard_block=64)
    codes, scales = ow.quantize_weight(oh.to_f32(w, "bf16"), oh.to_f32(lam, "bf16"), 64)
    ref = oh.from_f32(ow.linear_f32(oh.to_f32(x, "bf16"), codes, scales, oh.to_f32(lam, "bf16"), None, 64), "bf16")
    assert np.array_equal(host(qkv), ref)
    v = qkv[:, (hq + hk) * D:].clone()
    q, k = qkv[:, :hq * D].unflatten(1, (hq, D)), qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    pos = rng.integers(0, 64, (T, 3)).astype(np.int32)
    wq = weights(rng, D, "bf16")
    w4.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), dims, dev(wq, "bf16"), dev(wq, "bf16"), inplace=True)
    check(q, ref[:, :hq * D].reshape(T, hq, D), pos, dims, "bf16", wq)
    check(k, ref[:, hq * D:(hq + hk) * D].reshape(T, hk, D), pos, dims, "bf16", wq)
    turned = host(qkv[:, :(hq + hk) * D])
    w4.hadamard_transform(qkv[:, :(hq + hk) * D], block=D, inplace=True)
    assert np.array_equal(host(qkv[:, :(hq + hk) * D]), oh.hadamard_transform(turned, D, "bf16"))
    assert torch.equal(qkv[:, (hq + hk) * D:], v)


def turned_units(w4, dims, layout, theta, shared, pos, D, sin_cos):
    """The rotation of (1, 0) and of (0, 1) in every pair, in f32: its outputs are the kernel's cosines and sines as
    they are.  Each is checked against 64 bits within ``sin_cos(value, largest angle of the token)``."""
    import torch
    table = orope.pair_table(dims, layout, shared)
    x = np.zeros((len(pos), 2, D), np.float32)
    for e0, e1, _, _ in table:
        x[:, 0, e0] = x[:, 1, e1] = 1.0
    y = host(w4.qk_norm_rope(torch.from_numpy(x).cuda(), None, torch.from_numpy(pos).cuda(), dims, norm=False,
                             theta=theta, layout=layout, shared_frequencies=shared)).astype(np.float64)
    ref, _ = orope.norm_rope(x, pos, dims, theta=theta, layout=layout, shared=shared, norm=False)
    far = np.zeros(len(pos))
    for _, _, a, ex in table:
        far = np.maximum(far, np.abs(pos[:, a].astype(np.float64)) * theta ** -ex)
    off = np.abs(y - ref) / sin_cos(np.abs(ref), far[:, None, None])
    at = np.unravel_index(np.argmax(off), off.shape)
    assert off[at] <= 1, f"D={D} axes={dims} {layout} theta={theta}: {off[at]:.1f} times the bound at {at}: {y[at]} for {ref[at]}"


# A cosine or sine of its own: sincospi 2 units in the last place (4 * 2^-24 of the value), the step from the argument
# that sincospi gets, rounded to float32, to the whole one half a unit (2^-24 of the value).  That step is at most pi 2^-25
# times the other of the two, whose own roundings and its square's half are below 4e-14.  The float64 angle: 6 * 2^-53
# of the token's largest.
def own_size(value, far):
    return 5 * 2.0 ** -24 * value + 4e-14 + 6 * 2.0 ** -53 * far


@pytest.mark.parametrize("layout", LAYOUTS)
def test_small_sines_and_cosines(w4, layout):
    """Sines and cosines next to multiples of a quarter turn are as accurate as their own size asks for, which the
    float32 rounding of the angle alone would not leave."""
    pos = np.concatenate([np.arange(-1000, 1001), [31, 355, 710, 103993]]).astype(np.int32)[:, None]
    for D, dims in ((64, [64]), (2, [2]), (34, [34]), (128, [126]), (512, [512])):
        turned_units(w4, dims, layout, 10000.0, False, pos, D, own_size)
    two = np.concatenate([pos, pos[::-1]], 1)
    turned_units(w4, [44, 20], layout, 10000.0, True, two, 64, own_size)


@pytest.mark.parametrize("theta", [0.5, 1e-2, 1e-4, 3e-7, 1e-8, 1e-12])
def test_theta_below_one(w4, theta):
    """Ladders of rising frequencies: the float64 angle is within 6 * 2^-53 of the token's largest here too.  Positions
    that put this bound, for the largest angle, at about 1e-3."""
    rng = np.random.default_rng(13)
    for D, dims, layout, shared in ((64, [64], "half", False), (48, [48], "interleaved", False), (80, [40, 32], "axis_half", False),
                                    (64, [16, 24, 24], "half", True), (2, [2], "interleaved", False), (34, [34], "half", True)):
        n = sum(dims) if shared else max(dims)
        top = theta ** -(1 - 2 / n)  # the largest frequency
        far = int(min(max(1e12 / top, 3), 2.0 ** 40))
        pos = rng.integers(-far, far + 1, (300, len(dims)))
        turned_units(w4, dims, layout, theta, shared, pos, D, own_size)


def walked(w4, T, hq, hk, D, dims, dtype, layout):
    """q and k partitions of T rows where workgroups make several passes: tokens next to every kind of border against
    the oracle, all of them against calls of 500 tokens (one pass per workgroup), bit for bit, and in place."""
    import torch
    tokens = passes(T, hq + hk, D, dims, layout, dtype)
    print(f"\nT={T} heads={hq}+{hk} D={D} axes={dims} {dtype} {layout}: {tokens} tokens per pass", flush=True)
    assert -(-T // tokens) > 1536, "more blocks of tokens than workgroups"
    rng = np.random.default_rng(T + D)
    g = torch.Generator(device="cuda").manual_seed(T + D)
    # a column before the heads and one behind them, a row behind the last token
    big = torch.full((T + 1, (hq + hk) * D + 2), 5.0, dtype=tdtype(dtype), device="cuda")
    big[:T, 1:-1] = torch.randn((T, (hq + hk) * D), generator=g, device="cuda") * 1.5
    heads = big[:T, 1:-1].unflatten(1, (hq + hk, D))
    q, k = heads[:, :hq], heads[:, hq:]
    wq, wk = weights(rng, D, dtype), weights(rng, D, dtype)
    pos = rng.integers(-500, 500, (T, len(dims)))
    pt, wqt, wkt = torch.from_numpy(pos.astype(np.int32)).cuda(), dev(wq, dtype), dev(wk, dtype)
    a, b = w4.qk_norm_rope(q, k, pt, dims, wqt, wkt, layout=layout)
    step = 1536 * tokens
    some = np.unique(np.clip(np.concatenate([np.arange(30), np.arange(step - 30, step + 30), np.arange(T - 30, T),
                                             rng.integers(0, T, 100)]), 0, T - 1))
    at = torch.from_numpy(some).cuda()
    check(a[at], host(q[at]), pos[some], dims, dtype, wq, layout, what="q")
    check(b[at], host(k[at]), pos[some], dims, dtype, wk, layout, what="k")
    for t in range(0, T, 500):
        c, d = w4.qk_norm_rope(q[t:t + 500], k[t:t + 500], pt[t:t + 500], dims, wqt, wkt, layout=layout)
        assert torch.equal(c, a[t:t + 500]) and torch.equal(d, b[t:t + 500]), f"tokens {t} .. {t + 499}"
    w4.qk_norm_rope(q, k, pt, dims, wqt, wkt, layout=layout, inplace=True)
    assert torch.equal(q, a) and torch.equal(k, b)
    assert bool((big[:, 0] == 5).all() and (big[:, -1] == 5).all() and (big[T] == 5).all())


def passes(T, heads, D, dims, layout, dtype):
    """Tokens per pass: about six (token, head) items for each of a workgroup's lane groups, 1 to 8."""
    pairs = {"interleaved": [4], "half": [sum(dims) // 2], "axis_half": np.cumsum(dims) // 2}[layout]
    vector = D % 8 == 0 and all(p % 4 == 0 for p in pairs)
    lanes = D / 8 if vector else D / 4 if dtype == "f32" and 96 < D <= 128 else D / 8
    groups = 256 >> int(np.ceil(np.log2(np.ceil(lanes))))
    return min(max(6 * groups // heads, 1), 8, -(-T // 1536))


WALKS = [(20011, 3, 1, 64, [20, 2], "axis_half"), (26001, 1, 1, 128, [44, 42, 42], "axis_half"), (5003, 60, 4, 64, [20, 24], "half"),
         (13001, 24, 24, 24, [6, 10, 8], "axis_half"), (2003, 32, 2, 512, [250, 130], "half"), (8001, 8, 8, 256, [100, 152], "half")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", WALKS, ids=str)
def test_many_passes_of_staged_heads(w4, case, dtype):
    """Heads of whole 16-byte chunks whose pairs are not in whole fours: through LDS in 16 bits, element by element in f32
    (two items in flight where D is 128).  Passes of 8, 3 and 1 tokens."""
    walked(w4, *case[:-1], dtype, case[-1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", [(20011, 3, 2, 66, [30, 20], "half"), (20001, 2, 1, 126, [60, 66], "interleaved"), (2003, 40, 40, 90, [30, 60], "axis_half"),
                                  (13003, 3, 2, 64, [24, 40], "half"), (13001, 3, 1, 128, [44, 42, 42], "interleaved")], ids=str)
def test_many_passes_of_other_heads(w4, case, dtype):
    """The same for the element-wise forms and the vector path."""
    walked(w4, *case[:-1], dtype, case[-1])


@pytest.mark.parametrize("M", [5, 77])
def test_4bit_projection_then_norm_and_rotation(w4, M):
    """The chain of a fused q / k / v projection behind the 4-bit layer: its output against the oracle's gates, then q and
    k of that output normed and rotated in place, then rotated per head by the block Hadamard transform."""
    import torch
    import helpers as H
    from w4a4_bit_quantized_amd import synth
    rng = np.random.default_rng(M)
    K, hq, hk, D, dims = 512, 4, 2, 64, [16, 24, 24]
    N, qk = (hq + 2 * hk) * D, (hq + hk) * D
    lay = synth.make_layer("tiny", seed=M, M=M, K=K, N=N, R=32, B=64)
    weight, scales = H.oracle_weights(lay)
    qkv = w4.svdq_linear(H.to_dev_bf16(lay["x"]), H.device_layer(lay, weight, scales), hadamard_block=64)
    H.assert_gates(H.from_dev_bf16_f64(qkv), H.oracle_linear_rows(lay, weight, scales)[1], "4-bit projection")
    before = host(qkv)
    q, k = qkv[:, :hq * D].unflatten(1, (hq, D)), qkv[:, hq * D:qk].unflatten(1, (hk, D))
    pos = rng.integers(0, 64, (M, 3)).astype(np.int32)
    wq, wk = weights(rng, D, "bf16"), weights(rng, D, "bf16")
    w4.qk_norm_rope(q, k, torch.from_numpy(pos).cuda(), dims, dev(wq, "bf16"), dev(wk, "bf16"), inplace=True)
    check(q, before[:, :hq * D].reshape(M, hq, D), pos, dims, "bf16", wq)
    check(k, before[:, hq * D:qk].reshape(M, hk, D), pos, dims, "bf16", wk)
    turned = host(qkv[:, :qk])
    w4.hadamard_transform(qkv[:, :qk], block=D, inplace=True)
    assert np.array_equal(host(qkv[:, :qk]), oh.hadamard_transform(turned, D, "bf16"))
    assert np.array_equal(host(qkv[:, qk:]), before[:, qk:])
