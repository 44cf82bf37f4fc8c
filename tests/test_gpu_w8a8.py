"""GPU parity of the W8A8 layer (needs an MI355X) against ``oracle/w8a8.py``.

The quantizers perform the oracle's float32 operations (their two-part division is the correctly
rounded quotient), the integer sum is exact and the epilogue is the oracle's float32 operations in
the oracle's order, so codes, scales and outputs are all compared bit for bit.
"""

import numpy as np
import pytest

from oracle import hadamard as oh
from oracle import w8a8 as ow

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f16", "f32"]


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import w4a4_bit_quantized_amd as w
    w.load_library()
    return w


def dev(stored, dtype):
    import torch
    a = np.ascontiguousarray(stored)
    if dtype == "bf16":
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()
    return torch.from_numpy(a).cuda()


def host(t):
    """Stored values of a device tensor: uint16 bits for bf16, else the numpy dtype."""
    import torch
    t = t.detach().contiguous().cpu()
    return t.view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.numpy()


def tdtype(dtype):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]


def same_bits(got, ref, what=""):
    """Equal bit for bit, any NaN equal to any NaN."""
    got, ref = np.asarray(got), np.asarray(ref)
    assert got.shape == ref.shape and got.dtype == ref.dtype, (got.shape, got.dtype, ref.shape, ref.dtype)
    if got.dtype == np.uint16:
        bad = (got != ref) & ~(((got & 0x7FFF) > 0x7F80) & ((ref & 0x7FFF) > 0x7F80))
    else:
        u = {1: np.uint8, 2: np.uint16, 4: np.uint32}[got.dtype.itemsize]
        bad = got.view(u) != ref.view(u)
        if got.dtype.kind == "f":
            bad &= ~(np.isnan(got) & np.isnan(ref))
            bad &= ~((got == 0) & (ref == 0))  # the sign of a zero scale or sum is not part of the contract
    at = np.argwhere(bad)
    assert at.size == 0, f"{what}: {len(at)} of {got.size} differ, first at {at[:3].tolist()}"


def rows(rng, M, K, dtype, scale=1.0):
    """Tokens with outlier channels, as stored values."""
    x = rng.standard_normal((M, K)) * scale
    x[:, rng.permutation(K)[:max(1, K // 100)]] *= 20
    return oh.from_f32(x.astype(np.float32), dtype)


def factors(rng, K):
    return oh.from_f32(rng.uniform(0.5, 2.0, K).astype(np.float32), "bf16")


def check_quant(w4, x, dtype, lam, block, what, weight=False):
    import torch
    f = w4.w8a8_quantize_weight if weight else w4.w8a8_quantize_act
    q, s = f(dev(x, dtype), None if lam is None else dev(lam, "bf16"), hadamard_block=block)
    torch.cuda.synchronize()
    xf, lf = oh.to_f32(x, dtype), None if lam is None else oh.to_f32(lam, "bf16")
    qr, sr = (ow.quantize_weight if weight else ow.quantize_act)(xf, lf, block)
    same_bits(host(s), sr, f"{what} scales")
    same_bits(host(q), qr, f"{what} codes")


# K around every change of the kernel's thread and chunk counts, and past the register-resident rows
QUANT_K = [16, 48, 128, 2032, 2048, 2064, 4096, 4112, 6144, 6160, 8192, 8208, 12288, 12304, 16384, 16400, 20480]


@pytest.mark.parametrize("K", QUANT_K)
@pytest.mark.parametrize("M", [3, 1027])
def test_quantize_act_sizes(w4, M, K):
    rng = np.random.default_rng(K + M)
    M = M if M * K <= 6_000_000 else 1024 + 2  # enough rows for the many-row kernels
    dtype = DTYPES[(K // 16) % 3]
    check_quant(w4, rows(rng, M, K, dtype), dtype, factors(rng, K), 0, f"{M}x{K} {dtype}")
    if K % 128 == 0:
        check_quant(w4, rows(rng, min(M, 1030), K, "bf16"), "bf16", factors(rng, K), 128, f"{M}x{K} rotated")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block", [0, 16, 32, 64, 128])
@pytest.mark.parametrize("M", [1, 5, 1500])
def test_quantize_act_rotation_and_types(w4, dtype, block, M):
    rng = np.random.default_rng(M + block)
    for K in (640, 4480):
        check_quant(w4, rows(rng, M, K, dtype), dtype, factors(rng, K), block, f"{M}x{K} {dtype} B={block}")
    check_quant(w4, rows(rng, M, 384, dtype), dtype, None, block, f"{M}x384 {dtype} B={block} no smoothing")


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_weight(w4, dtype):
    rng = np.random.default_rng(5)
    for N, K, block in ((70, 272, 16), (33, 4224, 128), (5, 17408, 0), (1, 16, 0)):
        check_quant(w4, rows(rng, N, K, dtype, K ** -0.5), dtype, factors(rng, K), block, f"{N}x{K}", weight=True)
    check_quant(w4, rows(rng, 9, 96, dtype), dtype, None, 32, "no smoothing", weight=True)


@pytest.mark.parametrize("K,M", [(512, 8), (512, 1100), (16512, 8)])
@pytest.mark.parametrize("block", [0, 64])
def test_quantize_special_rows(w4, K, M, block):
    """Zero, tiny, non-finite and extreme rows among ordinary ones: every row on its own."""
    rng = np.random.default_rng(K + M)
    x = oh.to_f32(rows(rng, M, K, "f32"), "f32")
    x[0] = 0
    x[1] = 2.0 ** -105
    x[2, 3] = np.inf
    x[3, K - 1] = np.nan
    x[4] = 3e38
    x[5] = np.float32(2.0 ** -98) * rng.uniform(-1, 1, K).astype(np.float32)
    x[6] = 0
    x[6, 7] = -5.0
    x[M - 1, 1:] *= np.float32(2.0 ** -112)
    check_quant(w4, x, "f32", None, block, "no smoothing")
    check_quant(w4, x, "f32", factors(rng, K), block, "smoothing")


@pytest.mark.parametrize("K,M", [(256, 4), (256, 1100), (16640, 4)])
def test_quantize_extreme_factors(w4, K, M):
    """Smoothing factors outside the two-part division's range, zero, negative and non-finite ones."""
    rng = np.random.default_rng(K)
    x = rows(rng, M, K, "bf16")
    for values in ([2.0 ** -40, 1.0], [2.0 ** 50, 2.0 ** 50], [-1.5, 0.75], [0.0, 1.0], [np.nan, 1.0], [np.inf, 2.0],
                   [2.0 ** -32, 2.0 ** 32], [1e-39, 1.0]):
        lam = oh.from_f32(np.resize(np.array(values, np.float32), K), "bf16")
        check_quant(w4, x, "bf16", lam, 0, f"factors {values}")
        check_quant(w4, x, "bf16", lam, 32, f"factors {values} rotated")


def test_quantize_ties_and_divisions(w4):
    """Rows whose maximum is 127 put codes on integers and halves exactly; every bf16 mantissa as a
    smoothing factor against f32 values of random mantissas (the division has to round as IEEE's)."""
    rng = np.random.default_rng(11)
    x = np.arange(-254, 255, dtype=np.float32)[None, :508].repeat(4, 0) / 2
    x = np.concatenate([x, np.full((4, 4), 127, np.float32)], 1)
    check_quant(w4, x, "f32", None, 0, "ties")
    K = 4096
    lam = ((127 + rng.integers(-8, 9, K)) << 7 | np.arange(K) % 128).astype(np.uint16)
    bits = rng.integers(0, 1 << 23, (64, K)).astype(np.uint32) | (127 + rng.integers(-3, 4, (64, K)).astype(np.uint32)) << 23
    check_quant(w4, bits.view(np.float32), "f32", lam, 0, "divisions")
    check_quant(w4, bits.view(np.float32), "f32", lam, 16, "divisions rotated")


def codes(rng, *shape):
    return rng.integers(-127, 128, shape).astype(np.int8)


def check_gemm(w4, M, N, K, ydtype, bias, seed=0, out=None):
    import torch
    rng = np.random.default_rng(seed + M * 7 + N * 3 + K)
    qa, qw = codes(rng, M, K), codes(rng, N, K)
    qw[rng.integers(0, N)] = -128  # the most negative code is legal in a weight
    sa = rng.uniform(0.01, 0.1, M).astype(np.float32)
    sw = rng.uniform(0.001, 0.01, N).astype(np.float32)
    b = oh.from_f32(rng.uniform(-4, 4, N).astype(np.float32), "bf16") if bias else None
    y = w4.w8a8_gemm(torch.from_numpy(qa).cuda(), torch.from_numpy(sa).cuda(), torch.from_numpy(qw).cuda(),
                     torch.from_numpy(sw).cuda(), bias=None if b is None else dev(b, "bf16"), out=out,
                     out_dtype=tdtype(ydtype))
    torch.cuda.synchronize()
    ref = ow.gemm_f32(qa, sa, qw, sw, None if b is None else oh.to_f32(b, "bf16"))
    same_bits(host(y), oh.from_f32(ref, ydtype), f"{M}x{N}x{K} {ydtype}")


GEMM_SHAPES = [(330, 741, 64), (281, 434, 80), (350, 4044, 48), (4099, 4099, 64), (4090, 4100, 64), (1100, 4110, 96), (1, 1, 16), (1, 33, 64), (7, 200, 1040), (16, 256, 512), (17, 100, 528), (32, 64, 2048), (33, 130, 144),
               (64, 96, 4096), (65, 64, 128), (65, 1, 16), (100, 131, 272), (128, 4096, 256), (130, 9000, 400),
               (513, 3001, 128), (640, 4096, 1040), (1100, 8200, 144), (2048, 6200, 1552), (300, 40, 16400)]


@pytest.mark.parametrize("shape", GEMM_SHAPES)
def test_gemm_shapes(w4, shape):
    M, N, K = shape
    print(f"\ngemm {shape}", flush=True)
    check_gemm(w4, M, N, K, DTYPES[(M + N) % 3], bias=(M + K) % 2 == 0)


@pytest.mark.parametrize("tile", ["skinny", "32", "64x32", "64", "64x128", "64x128s4", "128", "128x192", "128x256", "256x192", "256"])
@pytest.mark.parametrize("shape", [(1, 16, 16), (16, 48, 128), (16, 4111, 400), (32, 65, 144), (32, 4130, 272), (32, 8200, 272), (64, 260, 2064)])
@pytest.mark.parametrize("ydtype", DTYPES)
def test_gemm_every_kernel(w4, hooks, tile, shape, ydtype):
    """Every kernel at sizes smaller than its tile, at odd sizes, and with K ending inside a K-step."""
    hooks.setenv("W8A8_GEMM_TILE", tile)
    print(f"\ntile {tile} {shape} {ydtype}", flush=True)
    check_gemm(w4, *shape, ydtype, bias=True)


@pytest.mark.parametrize("tile", ["32", "64x32", "64", "64x128", "64x128s4", "128", "128x192", "128x256", "256x192", "256"])
def test_gemm_tiled_larger(w4, hooks, tile):
    hooks.setenv("W8A8_GEMM_TILE", tile)
    for shape in ((300, 523, 1040), (513, 1032, 640), (257, 255, 16)):
        check_gemm(w4, *shape, "bf16", bias=False)


@pytest.mark.parametrize("tile", ["skinny", "32", "64x32", "64", "64x128", "64x128s4", "128", "128x192", "128x256", "256x192", "256"])
def test_gemm_rows_off_lines(w4, hooks, tile):
    """Rows that start anywhere in a 128-byte line (K modulo 128, operands at offsets of 16 bytes), in buffers
    of exactly their size."""
    import torch
    hooks.setenv("W8A8_GEMM_TILE", tile)
    rng = np.random.default_rng(len(tile))
    M, N = (29, 75) if tile == "skinny" else (131, 203)
    sa, sw = rng.uniform(0.01, 0.1, M).astype(np.float32), rng.uniform(0.001, 0.01, N).astype(np.float32)
    for K, oa, ob in ((16, 1, 0), (112, 0, 3), (128, 7, 0), (256, 0, 5), (384, 2, 6), (144, 0, 0), (1168, 3, 1), (1232, 0, 0),
                      (496, 5, 5), (2000, 0, 0), (1536, 4, 4), (4176, 0, 2)):
        qa, qw = codes(rng, M, K), codes(rng, N, K)
        put = lambda q, o: torch.cat([torch.full((16 * o,), 99, dtype=torch.int8), torch.from_numpy(q).flatten()]).cuda()[16 * o:].view(q.shape)
        y = w4.w8a8_gemm(put(qa, oa), torch.from_numpy(sa).cuda(), put(qw, ob), torch.from_numpy(sw).cuda(), out_dtype=torch.float32)
        same_bits(host(y), ow.gemm_f32(qa, sa, qw, sw, None), f"K={K} offsets {oa} {ob}")


def test_gemm_largest_sum(w4):
    """K at its maximum with every product 127 * 128: the int32 sum is within 2^31."""
    import torch
    from w4a4_bit_quantized_amd import binding
    K = binding.W8A8_MAX_K
    for M, N in ((3, 20), (80, 70)):
        qa = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
        qw = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        y = w4.w8a8_gemm(qa, torch.ones(M, device="cuda"), qw, torch.ones(N, device="cuda"), out_dtype=torch.float32)
        assert torch.equal(y.cpu(), torch.full((M, N), float(np.float32(-127 * 128 * K))))


@pytest.mark.parametrize("M,N", [(5, 40), (70, 137), (300, 264)])
@pytest.mark.parametrize("ydtype", DTYPES)
def test_gemm_into_a_partition(w4, M, N, ydtype):
    """An output partition of a wider matrix, aligned and not: nothing outside it is written."""
    import torch
    for start, width in ((16, N + 48), (3, N + 8), (4, N + 12), (2, N + 9)):
        big = torch.full((M + 2, width), 7.0, dtype=tdtype(ydtype), device="cuda")
        check_gemm(w4, M, N, 272, ydtype, True, out=big[1:M + 1, start:start + N])
        keep = torch.ones_like(big, dtype=torch.bool)
        keep[1:M + 1, start:start + N] = False
        assert bool((big[keep] == 7.0).all()), "columns or rows outside the partition were written"


@pytest.mark.parametrize("case", [(1, 512, 300, 0, "bf16", "bf16"), (20, 1040, 264, 16, "f16", "f16"),
                                  (48, 2048, 520, 128, "f32", "bf16"), (200, 640, 515, 64, "bf16", "f32"),
                                  (1030, 4224, 640, 32, "bf16", "bf16"), (64, 17408, 72, 128, "bf16", "bf16")])
def test_linear(w4, case):
    """The whole layer, 3-D input, a caller's workspace and a strided input view."""
    import torch
    M, K, N, block, xd, yd = case
    rng = np.random.default_rng(M)
    x, lam = rows(rng, M, K, xd), factors(rng, K)
    wf = rng.standard_normal((N, K)).astype(np.float32) * K ** -0.5
    qw, sw = ow.quantize_weight(wf, oh.to_f32(lam, "bf16"), block)
    b = oh.from_f32(rng.uniform(-1, 1, N).astype(np.float32), "bf16")
    layer = dict(qweight=torch.from_numpy(qw).cuda(), wscales=torch.from_numpy(sw).cuda(), smooth_factor=dev(lam, "bf16"),
                 bias=dev(b, "bf16"))
    ref = oh.from_f32(ow.linear_f32(oh.to_f32(x, xd), qw, sw, oh.to_f32(lam, "bf16"), oh.to_f32(b, "bf16"), block), yd)
    xt = dev(x, xd)
    y = w4.w8a8_linear(xt, layer, hadamard_block=block, out_dtype=tdtype(yd))
    same_bits(host(y), ref, "2-D")
    wide = torch.zeros((M, K + 24), dtype=xt.dtype, device="cuda")
    wide[:, 8:8 + K] = xt
    ws = torch.empty(w4.w8a8_linear_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    out = torch.empty((M, N), dtype=tdtype(yd), device="cuda")
    got = w4.w8a8_linear(wide[:, 8:8 + K], layer, hadamard_block=block, workspace=ws, out=out)
    assert got is out
    same_bits(host(out), ref, "strided input")
    if M % 2 == 0:
        y3 = w4.w8a8_linear(xt.view(2, M // 2, K), layer, hadamard_block=block, out_dtype=tdtype(yd))
        assert tuple(y3.shape) == (2, M // 2, N)
        same_bits(host(y3).reshape(M, N), ref, "3-D")


@pytest.mark.parametrize("K", [16, 144, 2048, 2064, 4096, 4112, 8192, 8208])
@pytest.mark.parametrize("xd", DTYPES)
def test_linear_one_token(w4, hooks, K, xd):
    """One token (one launch up to K = 8192): against the oracle and the two-launch layer, with and
    without smoothing, rotation and bias, at ragged channel counts, and with a row that counts as zero or NaN."""
    import torch
    rng = np.random.default_rng(K)
    for N, block, yd, special in ((1, 0, "bf16", 0), (37, 16, "f32", 0), (96, 128 if K % 128 == 0 else 0, "f16", 0),
                                  (40, 0, "f32", 1), (40, 16, "f32", 2),
                                  (4127, 0, "bf16", 0)):
        x, lam = rows(rng, 1, K, xd), factors(rng, K)
        if special:
            xf = oh.to_f32(x, xd).copy()
            if special == 1:
                xf[:] = 0
            else:
                xf[0, K // 2] = np.nan
            x = oh.from_f32(xf, xd)
        qw, sw = codes(rng, N, K), rng.uniform(0.001, 0.01, N).astype(np.float32)
        b = oh.from_f32(rng.uniform(-1, 1, N).astype(np.float32), "bf16") if block else None
        smooth = N != 1
        layer = dict(qweight=torch.from_numpy(qw).cuda(), wscales=torch.from_numpy(sw).cuda())
        if smooth:
            layer["smooth_factor"] = dev(lam, "bf16")
        if b is not None:
            layer["bias"] = dev(b, "bf16")
        ref = oh.from_f32(ow.linear_f32(oh.to_f32(x, xd), qw, sw, oh.to_f32(lam, "bf16") if smooth else None,
                                        None if b is None else oh.to_f32(b, "bf16"), block), yd)
        for mode in ("1", "0"):
            hooks.setenv("W8A8_ONE_LAUNCH", mode)
            y = w4.w8a8_linear(dev(x, xd), layer, hadamard_block=block, out_dtype=tdtype(yd))
            same_bits(host(y), ref, f"K={K} N={N} {xd} {yd} one launch {mode}")


@pytest.mark.parametrize("M", [2, 3, 4, 5])
@pytest.mark.parametrize("K", [16, 400, 2048, 4112, 6144, 8192])
def test_linear_few_tokens(w4, hooks, M, K):
    """A few tokens (one launch up to 4): strided input and output rows, a zero row and a NaN row among them, with and
    without smoothing, rotation and bias, against the oracle and the two-launch layer."""
    import torch
    rng = np.random.default_rng(M * K)
    for N, block, xd, yd, smooth in ((37, 16, "bf16", "f32", True), (300, 128 if K % 128 == 0 else 0, "f16", "bf16", False),
                                     (4099, 0, "f32", "f16", True)):
        x, lam = rows(rng, M, K, xd), factors(rng, K)
        xf = oh.to_f32(x, xd).copy()
        xf[M // 2] = 0
        if N == 37:
            xf[M - 1, K // 3] = np.nan
        x = oh.from_f32(xf, xd)
        qw, sw = codes(rng, N, K), rng.uniform(0.001, 0.01, N).astype(np.float32)
        b = oh.from_f32(rng.uniform(-1, 1, N).astype(np.float32), "bf16") if block else None
        layer = dict(qweight=torch.from_numpy(qw).cuda(), wscales=torch.from_numpy(sw).cuda(),
                     smooth_factor=dev(lam, "bf16") if smooth else None, bias=None if b is None else dev(b, "bf16"))
        ref = oh.from_f32(ow.linear_f32(xf, qw, sw, oh.to_f32(lam, "bf16") if smooth else None,
                                        None if b is None else oh.to_f32(b, "bf16"), block), yd)
        wide = torch.zeros((M, K + 24), dtype=tdtype(xd), device="cuda")
        wide[:, 8:8 + K] = dev(x, xd)
        for mode in ("1", "0"):
            hooks.setenv("W8A8_ONE_LAUNCH", mode)
            big = torch.full((M + 1, N + 5), 7.0, dtype=tdtype(yd), device="cuda")
            y = w4.w8a8_linear(wide[:, 8:8 + K], layer, hadamard_block=block, out=big[:M, 3:3 + N])
            same_bits(host(y), ref, f"M={M} K={K} N={N} {xd} {yd} one launch {mode}")
            big[:M, 3:3 + N] = 7.0
            assert bool((big == 7.0).all()), "elements around the output were written"


def test_linear_one_token_extreme_factors(w4):
    """Smoothing factors outside the two-part division's range, in the one-launch layer."""
    import torch
    rng = np.random.default_rng(1)
    K, N = 512, 33
    x = rows(rng, 1, K, "bf16")
    qw, sw = codes(rng, N, K), np.ones(N, np.float32)
    for values in ([2.0 ** -40, 1.0], [2.0 ** 50, 2.0], [0.0, 1.0], [np.inf, 2.0], [-3.0, 1.0]):
        lam = oh.from_f32(np.resize(np.array(values, np.float32), K), "bf16")
        y = w4.w8a8_linear(dev(x, "bf16"), dict(qweight=torch.from_numpy(qw).cuda(), wscales=torch.from_numpy(sw).cuda(),
                                                smooth_factor=dev(lam, "bf16")), out_dtype=torch.float32)
        same_bits(host(y), ow.linear_f32(oh.to_f32(x, "bf16"), qw, sw, oh.to_f32(lam, "bf16")), f"factors {values}")


def test_linear_nonfinite_rows_stay_alone(w4):
    """A row with an infinity or a NaN is NaN throughout; the other rows are as without it."""
    import torch
    rng = np.random.default_rng(2)
    for M in (6, 100):
        K, N = 256, 72
        x = dev(rows(rng, M, K, "bf16"), "bf16")
        qw, sw = w4.w8a8_quantize_weight(dev(rows(rng, N, K, "bf16"), "bf16"))
        layer = dict(qweight=qw, wscales=sw)
        clean = w4.w8a8_linear(x, layer)
        x[2, 5], x[4, 0] = float("inf"), float("nan")
        y = w4.w8a8_linear(x, layer)
        assert bool(y[[2, 4]].isnan().all())
        rest = [r for r in range(M) if r not in (2, 4)]
        assert torch.equal(y[rest], clean[rest])


def test_empty_and_refused_calls(w4):
    import torch
    e = dict(qweight=torch.zeros((8, 64), dtype=torch.int8, device="cuda"), wscales=torch.zeros(8, device="cuda"))
    assert tuple(w4.w8a8_linear(torch.zeros((0, 64), device="cuda"), e).shape) == (0, 8)
    n = dict(qweight=e["qweight"][:0], wscales=e["wscales"][:0])
    assert tuple(w4.w8a8_linear(torch.zeros((3, 64), device="cuda"), n).shape) == (3, 0)
    x = torch.zeros((4, 72), device="cuda", dtype=torch.bfloat16)
    with pytest.raises(w4.W4A4Error, match="ERR_ALIGN"):
        w4.w8a8_linear(x[:, 4:68], e)
    with pytest.raises(w4.W4A4Error, match="ERR_SHAPE"):
        w4.w8a8_linear(torch.zeros((4, 68), device="cuda")[:, :64], e)
    with pytest.raises(w4.W4A4Error, match="ERR_SHAPE"):
        w4.w8a8_quantize_act(torch.zeros((4, 40), device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        w4.w8a8_linear(x[:, :64].contiguous(), e, workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="qweight"):
        w4.w8a8_linear(torch.zeros((4, 80), device="cuda"), e)
    with pytest.raises(TypeError, match="qweight"):
        w4.w8a8_linear(torch.zeros((4, 64), device="cuda"), dict(e, qweight=e["qweight"].to(torch.uint8)))
    with pytest.raises(ValueError, match="out"):
        w4.w8a8_linear(torch.zeros((4, 64), device="cuda"), e, out=torch.zeros((4, 9), device="cuda"))


def test_graph_replay_and_side_stream(w4):
    """Captured once, replayed on changed inputs between eager calls; and on a stream of its own."""
    import torch
    rng = np.random.default_rng(9)
    for M in (8, 300):
        K, N = 1040, 328
        x = dev(rows(rng, M, K, "bf16"), "bf16")
        qw, sw = w4.w8a8_quantize_weight(dev(rows(rng, N, K, "bf16"), "bf16"))
        layer = dict(qweight=qw, wscales=sw, smooth_factor=dev(factors(rng, K), "bf16"))
        ws = torch.empty(w4.w8a8_linear_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
        out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        w4.w8a8_linear(x, layer, hadamard_block=16, workspace=ws, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w4.w8a8_linear(x, layer, hadamard_block=16, workspace=ws, out=out)
        for _ in range(4):
            x.copy_(dev(rows(rng, M, K, "bf16"), "bf16"))
            ref = w4.w8a8_linear(x, layer, hadamard_block=16)
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            y = w4.w8a8_linear(x, layer, hadamard_block=16)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, ref)


def test_two_streams_and_one_token_graph(w4):
    """Calls on two streams at once, each with a workspace of its own, among them one-token calls; two captured
    one-token calls replayed in turn with eager ones between; the same input for several layers."""
    import torch
    rng = np.random.default_rng(21)
    K = 1040
    x1, x2 = dev(rows(rng, 1, K, "bf16"), "bf16"), dev(rows(rng, 700, K, "bf16"), "bf16")
    layers = []
    for N in (328, 1037):
        qw, sw = w4.w8a8_quantize_weight(dev(rows(rng, N, K, "bf16"), "bf16"))
        layers.append(dict(qweight=qw, wscales=sw, smooth_factor=dev(factors(rng, K), "bf16")))
    want = [[w4.w8a8_linear(x, l, hadamard_block=16) for l in layers] for x in (x1, x2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for turn in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for l in layers:
                    got[i].append([w4.w8a8_linear(x, l, hadamard_block=16) for x in (x1, x2)])
    torch.cuda.synchronize()
    for g in got:
        for j, ys in enumerate(g):
            for y, w in zip(ys, (want[0][j % 2], want[1][j % 2])):
                assert torch.equal(y, w)
    ws = torch.empty(w4.w8a8_linear_workspace_bytes(1, K), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(w) for w in want[0]], []
    for l, o in zip(layers, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w4.w8a8_linear(x1, l, hadamard_block=16, workspace=ws, out=o)
        graphs.append(g)
    for _ in range(4):
        x1.copy_(dev(rows(rng, 1, K, "bf16"), "bf16"))
        ref = [w4.w8a8_linear(x1, l, hadamard_block=16) for l in layers]
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, ref))


def test_layer_object(w4):
    """W8A8Linear: quantized once from a weight, called with and without an output."""
    import torch
    from w4a4_bit_quantized_amd import checkpoint
    rng = np.random.default_rng(21)
    K, N = 256, 48
    w, lam = rows(rng, N, K, "bf16", K ** -0.5), factors(rng, K)
    b = oh.from_f32(rng.uniform(-1, 1, N).astype(np.float32), "bf16")
    layer = checkpoint.W8A8Linear.from_weight(dev(w, "bf16"), dev(lam, "bf16"), dev(b, "bf16"), hadamard_block=32)
    qw, sw = ow.quantize_weight(oh.to_f32(w, "bf16"), oh.to_f32(lam, "bf16"), 32)
    x = rows(rng, 12, K, "bf16")
    ref = ow.linear_f32(oh.to_f32(x, "bf16"), qw, sw, oh.to_f32(lam, "bf16"), oh.to_f32(b, "bf16"), 32)
    same_bits(host(layer(dev(x, "bf16"))), oh.from_f32(ref, "bf16"))
    out = torch.empty((12, N), dtype=torch.float32, device="cuda")
    assert layer(dev(x, "bf16"), out=out) is out
    same_bits(host(out), ref)


def special_rows(rng, K, dtype):
    """Forty rows as stored: ordinary ones of several sizes, zeros, tiny, huge, non-finite, one element alone."""
    xf = oh.to_f32(rows(rng, 40, K, dtype), dtype).copy()
    xf[8:16] *= np.float32(2.0 ** -9)
    xf[0] = 0
    xf[1] = 2.0 ** -105  # (0 in f16)
    xf[2, 3] = np.inf
    xf[3, K - 1] = np.nan
    xf[4] = 3e38 if dtype != "f16" else 65504.0
    xf[5] = 0
    xf[5, 7] = -5.0
    xf[6, 1:] *= np.float32(2.0 ** -112)
    xf[7, :-1] = 0
    with np.errstate(over="ignore"):
        return oh.from_f32(xf, dtype)


def many_rows(w4, rng, x, dtype, lam, block, M, pad=0):
    """M tokens drawn from the rows of ``x`` (in a matrix ``pad`` columns wider), quantized into the middle of larger
    buffers: every row is its oracle row wherever it sits, and nothing around the outputs is written."""
    import torch
    K = x.shape[1]
    idx = rng.integers(0, len(x), M)
    assert all(set(idx[p::2]) >= set(range(8)) for p in (0, 1)), "special rows in both places of a pair"
    wide = torch.empty((M, K + pad), dtype=tdtype(dtype), device="cuda")
    xt = wide[:, :K]
    xt.copy_(dev(x, dtype)[torch.from_numpy(idx).cuda()])
    lt = None if lam is None else dev(lam, "bf16")
    q = torch.full((M + 2, K), 77, dtype=torch.int8, device="cuda")
    s = torch.full((M + 2,), 77.0, device="cuda")
    st = w4.load_library().w8a8_quantize_act(xt.data_ptr(), K + pad, DTYPES.index(dtype), None if lt is None else lt.data_ptr(),
                                             M, K, block, q[1:].data_ptr(), s[1:].data_ptr(),
                                             torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    what = f"{M}x{K} {dtype} B={block}"
    qr, sr = ow.quantize_act(oh.to_f32(x, dtype), None if lam is None else oh.to_f32(lam, "bf16"), block)
    got_q, got_s = host(q), host(s)
    same_bits(got_s[1:-1], sr[idx], f"{what} scales")
    same_bits(got_q[1:-1], qr[idx], f"{what} codes")
    assert (got_q[[0, -1]] == 77).all() and (got_s[[0, -1]] == 77).all(), f"{what}: rows around the outputs were written"


# from 2048 rows on a workgroup takes two rows per pass, one chunk of 8 columns per thread up to 8192 columns, two up to
# 16384; 256 to 6144 workgroups, so that 4099 rows (20000 at 208 columns) are several passes for each
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [208, 1040, 4224, 8192, 8208, 8320, 16384])
def test_quantize_two_rows_per_pass(w4, K, dtype):
    rng = np.random.default_rng(K)
    x, lam = special_rows(rng, K, dtype), factors(rng, K)
    print(f"\nK={K} {dtype}", flush=True)
    for block in (0, 16, 32, 64, 128):
        if block == 0 or K % block == 0:
            for M in (2047, 2048, 2049):
                many_rows(w4, rng, x, dtype, lam, block, M)
    many_rows(w4, rng, x, dtype, None, 16, 4099, pad=24)
    many_rows(w4, rng, x, dtype, lam, 0, 4099 if K > 208 else 20001)


@pytest.mark.parametrize("K", [256, 8320])
def test_quantize_two_rows_extreme_factors(w4, K):
    """Smoothing factors outside the two-part division's range, zero, negative and non-finite ones, in two rows per pass."""
    rng = np.random.default_rng(K)
    x = special_rows(rng, K, "bf16")
    for values in ([2.0 ** -40, 1.0], [2.0 ** 50, 2.0 ** 50], [-1.5, 0.75], [0.0, 1.0], [np.nan, 1.0], [np.inf, 2.0], [1e-39, 1.0]):
        lam = oh.from_f32(np.resize(np.array(values, np.float32), K), "bf16")
        many_rows(w4, rng, x, "bf16", lam, 0, 2049)
        many_rows(w4, rng, x, "bf16", lam, 32, 2049)


def test_linear_two_rows_per_pass(w4):
    """The layer over the two-row quantizer: its row count is odd, and a workgroup takes several pairs."""
    import torch
    rng = np.random.default_rng(21)
    M, K, N = 2051, 4224, 136
    x, lam = rows(rng, M, K, "bf16"), factors(rng, K)
    qw, sw = codes(rng, N, K), rng.uniform(0.001, 0.01, N).astype(np.float32)
    y = w4.w8a8_linear(dev(x, "bf16"), dict(qweight=torch.from_numpy(qw).cuda(), wscales=torch.from_numpy(sw).cuda(),
                                            smooth_factor=dev(lam, "bf16")), hadamard_block=128)
    ref = ow.linear_f32(oh.to_f32(x, "bf16"), qw, sw, oh.to_f32(lam, "bf16"), None, 128)
    same_bits(host(y), oh.from_f32(ref, "bf16"), "layer of 2051 tokens")


def test_numbers_past_32_bits_are_refused(w4):
    """A block or an axis that only fits after its upper bits are lost is no valid one."""
    import torch
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    layer = dict(qweight=torch.ones((8, 64), dtype=torch.int8, device="cuda"), wscales=torch.ones(8, device="cuda"))
    q = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for far in (2 ** 32, -2 ** 32, 2 ** 40):
        for call in (lambda: w4.w8a8_quantize_act(x, hadamard_block=far + 64), lambda: w4.w8a8_quantize_weight(x, hadamard_block=far),
                     lambda: w4.w8a8_linear(x, layer, hadamard_block=far + 16), lambda: w4.hadamard_transform(x, block=far + 64),
                     lambda: w4.qk_norm_rope(q, None, pos, [far + 32, 32]), lambda: w4.qk_norm_rope(q, None, pos, [32, far])):
            with pytest.raises((ValueError, w4.W4A4Error)):
                call()
