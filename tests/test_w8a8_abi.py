"""CPU tests of the W8A8 and qk_norm_rope entry points: arguments are rejected before any launch (no GPU
is touched), and the binding's checks run before the library call."""

import ctypes
import os

import pytest

import w4a4_bit_quantized_amd as w4
from w4a4_bit_quantized_amd import binding

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED = 0, 1, 2, 3, 4
P = 0x10000  # a fake, well-aligned device address; never dereferenced by the validation paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        from w4a4_bit_quantized_amd import build
        build.build()
    return w4.load_library()


@pytest.mark.parametrize("name", ["w8a8_quantize_act", "w8a8_quantize_weight"])
def test_quantize_validation(lib, name):
    def f(x=P, ld=64, dt=0, lam=P, M=4, K=64, hb=0, q=P, s=P):
        return getattr(lib, name)(x, ld, dt, lam, M, K, hb, q, s, None)
    assert f(K=40) == ERR_SHAPE and f(K=0) == ERR_SHAPE and f(K=-16) == ERR_SHAPE
    assert f(M=-1) == ERR_SHAPE and f(M=1 << 31) == ERR_SHAPE
    assert f(ld=48) == ERR_SHAPE and f(ld=68) == ERR_SHAPE
    assert f(K=48, ld=48, hb=32) == ERR_SHAPE
    assert f(hb=8) == ERR_UNSUPPORTED and f(hb=256) == ERR_UNSUPPORTED and f(hb=-16) == ERR_UNSUPPORTED
    assert f(dt=3) == ERR_UNSUPPORTED and f(dt=-1) == ERR_UNSUPPORTED
    big = binding.W8A8_MAX_K + 16
    assert f(K=big, ld=big) == ERR_UNSUPPORTED
    assert f(M=0, x=None, lam=None, q=None, s=None) == OK
    assert f(x=None) == ERR_NULL and f(q=None) == ERR_NULL and f(s=None) == ERR_NULL
    assert f(x=P + 8) == ERR_ALIGN and f(lam=P + 2) == ERR_ALIGN and f(q=P + 4) == ERR_ALIGN and f(s=P + 2) == ERR_ALIGN


def test_gemm_validation(lib):
    def f(qa=P, sa=P, qw=P, sw=P, b=None, M=4, N=8, K=64, y=P, ldy=None, dt=0):
        return lib.w8a8_gemm(qa, sa, qw, sw, b, M, N, K, y, max(N, 0) if ldy is None else ldy, dt, None)
    assert f(K=72) == ERR_SHAPE and f(M=-1) == ERR_SHAPE and f(N=-1) == ERR_SHAPE and f(ldy=7) == ERR_SHAPE
    assert f(M=(1 << 31) - 1, N=1 << 20) == ERR_SHAPE  # more output tiles than a launch has workgroups
    assert f(dt=3) == ERR_UNSUPPORTED and f(K=binding.W8A8_MAX_K + 16) == ERR_UNSUPPORTED
    assert f(M=0, qa=None, y=None) == OK and f(N=0, qw=None) == OK
    for k in ("qa", "sa", "qw", "sw", "y"):
        assert f(**{k: None}) == ERR_NULL
    assert f(qa=P + 8) == ERR_ALIGN and f(qw=P + 8) == ERR_ALIGN and f(sa=P + 2) == ERR_ALIGN and f(sw=P + 1) == ERR_ALIGN
    assert f(b=P + 1) == ERR_ALIGN and f(y=P + 1) == ERR_ALIGN and f(y=P + 2, dt=2) == ERR_ALIGN


def test_linear_validation(lib):
    assert lib.w8a8_linear_workspace_bytes(3, 64) == 256 + 256
    assert lib.w8a8_linear_workspace_bytes(100, 1040) == 104192 + 512
    assert lib.w8a8_linear_workspace_bytes(-1, 64) == 0 and lib.w8a8_linear_workspace_bytes(4, 40) == 0
    assert lib.w8a8_linear_workspace_bytes(1 << 31, 64) == 0

    def f(x=P, ld=64, xd=0, qw=P, sw=P, lam=P, b=None, M=4, N=8, K=64, hb=0, y=P, ldy=8, yd=0, ws=P, wsb=1 << 20):
        return lib.w8a8_linear(x, ld, xd, qw, sw, lam, b, M, N, K, hb, y, ldy, yd, ws, wsb, None)
    assert f(K=40) == ERR_SHAPE and f(ld=56) == ERR_SHAPE and f(ldy=4) == ERR_SHAPE and f(N=-1) == ERR_SHAPE
    assert f(wsb=511) == ERR_SHAPE
    assert f(xd=5) == ERR_UNSUPPORTED and f(yd=5) == ERR_UNSUPPORTED and f(hb=3) == ERR_UNSUPPORTED
    assert f(M=0, x=None, ws=None) == OK and f(N=0, qw=None, ws=None, ldy=0) == OK
    assert f(ws=None) == ERR_NULL and f(x=None) == ERR_NULL and f(qw=None) == ERR_NULL and f(y=None) == ERR_NULL
    assert f(ws=P + 128) == ERR_ALIGN and f(x=P + 8) == ERR_ALIGN and f(b=P + 1) == ERR_ALIGN


def test_sizes_that_pass_32_and_64_bits(lib):
    """Row counts whose padded or strided successors pass 2^31, grids past 2^32 threads, and byte offsets past
    2^63 are refused; one row may have any stride."""
    rows = 1 << 28
    q = lambda M, ld: lib.w8a8_quantize_act(P, ld, 0, None, M, 64, 0, P, P + 2, None)
    assert q(rows, 64) == ERR_ALIGN and q(rows + 1, 64) == ERR_SHAPE and q((1 << 31) - 1, 64) == ERR_SHAPE
    assert q(2, 1 << 32) == ERR_ALIGN and q(2, (1 << 32) + 8) == ERR_SHAPE and q(1, 1 << 60) == ERR_ALIGN
    g = lambda M, N, ldy: lib.w8a8_gemm(P, P + 2, P, P, None, M, N, 16, P, ldy, 0, None)
    assert g(rows, 512, 512) == ERR_ALIGN and g(rows, 513, 513) == ERR_SHAPE and g(rows + 1, 1, 1) == ERR_SHAPE
    assert g(1, rows, rows) == ERR_ALIGN and g(1, rows + 1, rows + 1) == ERR_SHAPE and g(1 << 19, 1 << 19, 1 << 19) == ERR_SHAPE
    assert g(2, 8, (1 << 32) + 1) == ERR_SHAPE and g(1, 8, 1 << 60) == ERR_ALIGN
    f = lambda M, N, ldx, ldy: lib.w8a8_linear(P, ldx, 0, P, P + 2, None, None, M, N, 16, 0, P, ldy, 0, P, 1 << 40, None)
    assert f(rows, 512, 16, 512) == ERR_ALIGN and f(rows, 513, 16, 513) == ERR_SHAPE and f(rows + 1, 1, 16, 1) == ERR_SHAPE
    assert f(2, 8, (1 << 32) + 8, 8) == ERR_SHAPE and f(1, 8, 1 << 60, 8) == ERR_ALIGN
    assert lib.w8a8_linear_workspace_bytes(rows, 16) > 0 and lib.w8a8_linear_workspace_bytes(rows + 1, 16) == 0
    far = dict(T=(1 << 31) - 1, q=_heads(ts=1 << 29, w=P + 1, yts=512))
    assert _rope(lib, **far) == ERR_ALIGN
    far["q"].x_token_stride = 1 << 30
    assert _rope(lib, **far) == ERR_SHAPE
    assert _rope(lib, q=_heads(heads=1 << 15, hs=1 << 40, w=P + 1, yts=1 << 21)) == ERR_ALIGN
    assert _rope(lib, T=(1 << 31) - 1, q=_heads(yts=1 << 40, w=P + 1)) == ERR_SHAPE


def test_outputs_on_top_of_inputs(lib):
    f = lambda M: lib.w8a8_linear(P, 64, 0, P, P, None, None, M, 64, 64, 0, P, 64, 0, P, 1 << 20, None)
    assert f(4) == ERR_SHAPE and f(1) == ERR_SHAPE and f(0) == OK
    side = lambda **kw: _heads(w=P + 1, **kw)
    assert _rope(lib, q=side(), k=side()) == ERR_SHAPE                      # both outputs in one place
    assert _rope(lib, q=side(x=P, y=P), k=side(x=P, y=P)) == ERR_SHAPE      # q and k the same tensor, in place
    assert _rope(lib, q=side(), k=side(y=P + 0x200000)) == ERR_ALIGN        # the same input twice is fine


def _heads(x=P, ts=512, hs=64, heads=8, w=None, y=P + 0x100000, yts=512, yhs=64):
    return binding.Heads(x, ts, hs, heads, w, y, yts, yhs)


def _rope(lib, q=None, k=None, pos=P, T=4, D=64, dims=(64,), layout=0, flags=1, theta=1e4, eps=1e-6, dt=0, axes=None):
    q = _heads() if q is None else q
    arr = (ctypes.c_int32 * max(len(dims), 1))(*dims)
    return lib.w4a4_qk_norm_rope(ctypes.byref(q) if q else None, ctypes.byref(k) if k else None, pos, T, D,
                                 len(dims) if axes is None else axes, arr, layout, flags, theta, eps, dt, None)


def test_rope_validation(lib):
    r = lambda **kw: _rope(lib, **kw)
    assert r(dt=3) == ERR_UNSUPPORTED and r(layout=3) == ERR_UNSUPPORTED and r(layout=-1) == ERR_UNSUPPORTED
    assert r(flags=8) == ERR_UNSUPPORTED and r(D=514) == ERR_UNSUPPORTED and r(dims=(2,) * 9) == ERR_UNSUPPORTED
    assert r(T=-1) == ERR_SHAPE and r(D=0) == ERR_SHAPE and r(D=63) == ERR_SHAPE and r(axes=-1) == ERR_SHAPE
    assert r(dims=(66,)) == ERR_SHAPE and r(dims=(32, 34)) == ERR_SHAPE and r(dims=(3,)) == ERR_SHAPE and r(dims=(-2, 64)) == ERR_SHAPE
    for theta in (0.0, -1.0, float("inf"), float("nan")):
        assert r(theta=theta) == ERR_SHAPE
    for eps in (-1e-6, float("inf"), float("nan")):
        assert r(eps=eps) == ERR_SHAPE
    assert r(T=0, pos=None, q=_heads(x=None, y=None)) == OK
    assert r(q=_heads(heads=0, x=None, y=None)) == OK
    assert r(pos=None) == ERR_NULL and r(q=_heads(x=None)) == ERR_NULL and r(k=_heads(y=None)) == ERR_NULL
    assert lib.w4a4_qk_norm_rope(None, None, P, 4, 64, 0, None, 0, 1, 1e4, 1e-6, 0, None) == ERR_NULL
    assert lib.w4a4_qk_norm_rope(ctypes.byref(_heads()), None, P, 4, 64, 1, None, 0, 1, 1e4, 1e-6, 0, None) == ERR_NULL
    assert r(q=_heads(x=P + 1)) == ERR_ALIGN and r(q=_heads(y=P + 1)) == ERR_ALIGN and r(q=_heads(w=P + 1)) == ERR_ALIGN
    assert r(q=_heads(x=P + 2), dt=2) == ERR_ALIGN and r(pos=P + 2) == ERR_ALIGN and r(pos=P + 4, flags=5) == ERR_ALIGN


def test_rope_strides(lib):
    r = lambda **kw: _rope(lib, T=kw.pop("T", 4), q=_heads(**kw))
    assert r(heads=-1) == ERR_SHAPE and r(heads=1 << 16) == ERR_SHAPE
    assert r(ts=-512) == ERR_SHAPE and r(yhs=-64) == ERR_SHAPE and r(ts=1 << 41) == ERR_SHAPE
    assert r(yhs=63) == ERR_SHAPE                       # heads overlap
    assert r(yts=511) == ERR_SHAPE                      # tokens overlap
    assert r(yts=0, yhs=0) == ERR_SHAPE
    assert r(yts=32, yhs=256) == ERR_SHAPE              # neither heads in tokens nor tokens in heads
    assert r(x=P, y=P, yts=1024) == ERR_SHAPE           # in place needs equal strides
    assert r(x=P, y=P, hs=64, yhs=128, yts=1024, ts=1024) == ERR_SHAPE
    # accepted sizes reach the alignment check (an odd weight address), after every size check
    odd = dict(w=P + 1)
    assert r(**odd) == ERR_ALIGN
    assert r(yts=64, yhs=4 * 64, **odd) == ERR_ALIGN    # (heads, tokens, head_dim) output
    assert r(ts=512, hs=0, **odd) == ERR_ALIGN          # a broadcast head is read again
    assert r(x=P, y=P, **odd) == ERR_ALIGN              # in place
    assert r(heads=1, yhs=0, hs=0, **odd) == ERR_ALIGN  # one head: its stride does not matter
    assert r(T=1, yts=0, ts=0, **odd) == ERR_ALIGN
    assert r(x=P, y=P, T=1, ts=512, yts=7, **odd) == ERR_ALIGN


def test_constants_match_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w4a4.h")).read()
    for name, value in (("W8A8_MAX_K", binding.W8A8_MAX_K), ("W8A8_MAX_ROWS", "(1 << 28)"), ("W4A4_ROPE_MAX_HEAD_DIM", binding.ROPE_MAX_HEAD_DIM),
                        ("W4A4_ROPE_MAX_AXES", binding.ROPE_MAX_AXES), ("W4A4_ROPE_NORM", binding.ROPE_NORM),
                        ("W4A4_ROPE_SHARED_FREQUENCIES", binding.ROPE_SHARED_FREQUENCIES),
                        ("W4A4_ROPE_POSITIONS_I64", binding.ROPE_POSITIONS_I64),
                        ("W4A4_ROPE_INTERLEAVED", binding.ROPE_LAYOUTS["interleaved"]),
                        ("W4A4_ROPE_HALF", binding.ROPE_LAYOUTS["half"]),
                        ("W4A4_ROPE_AXIS_HALF", binding.ROPE_LAYOUTS["axis_half"])):
        assert f"#define {name} {value}\n" in text
    # the largest int32 sum: K * 127 * 128 < 2^31, and the next K that the layer could take overflows
    assert binding.W8A8_MAX_K % 16 == 0 and binding.W8A8_MAX_K * 127 * 128 < 2 ** 31


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        w4.w8a8_linear(x, dict(qweight=torch.zeros(8, 64, dtype=torch.int8), wscales=torch.zeros(8)))
    with pytest.raises(ValueError, match="device tensor"):
        w4.w8a8_gemm(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4), torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8))
    with pytest.raises(ValueError, match="device tensor"):
        w4.qk_norm_rope(torch.zeros(4, 2, 64), None, torch.zeros(4, 1, dtype=torch.int32), [64])
    with pytest.raises(TypeError, match="torch tensor"):
        w4.w8a8_quantize_act([1, 2])


def test_heads_view():
    import torch
    v = binding._heads_view
    assert v(torch.zeros(5, 3, 8), "q") == (5, 3, 8, 24, 8)
    assert v(torch.zeros(2, 5, 3, 8), "q") == (10, 3, 8, 24, 8)
    assert v(torch.zeros(2, 1, 3, 8), "q") == (2, 3, 8, 24, 8)
    assert v(torch.zeros(5, 100)[:, 8:32].view(5, 3, 8), "q") == (5, 3, 8, 100, 8)
    assert v(torch.zeros(3, 5, 8).transpose(0, 1), "q") == (5, 3, 8, 8, 40)
    with pytest.raises(ValueError, match="flatten"):
        v(torch.zeros(2, 9, 3, 8)[:, :5], "q")
    with pytest.raises(ValueError, match="dense"):
        v(torch.zeros(5, 3, 16)[..., ::2], "q")
    with pytest.raises(ValueError, match="must be"):
        v(torch.zeros(5, 24), "q")


def test_check_layer_w8a8():
    import torch
    from w4a4_bit_quantized_amd import checkpoint as c
    t = dict(qweight=torch.zeros(8, 64, dtype=torch.int8), wscales=torch.zeros(8))
    assert c.check_layer_w8a8(t) == (8, 64)
    assert c.check_layer_w8a8(dict(t, smooth_factor=torch.zeros(64, dtype=torch.bfloat16), bias=None)) == (8, 64)
    for bad in (dict(qweight=t["qweight"]), dict(t, qweight=torch.zeros(8, 64, dtype=torch.uint8)),
                dict(t, wscales=torch.zeros(9)), dict(t, qweight=torch.zeros(8, 40, dtype=torch.int8)),
                dict(t, bias=torch.zeros(8)), dict(t, smooth_factor=torch.zeros(63, dtype=torch.bfloat16)),
                dict(t, qweight=torch.zeros(8, dtype=torch.int8))):
        with pytest.raises(c.ContractError):
            c.check_layer_w8a8(bad)


def test_rope_output_on_the_other_input(lib):
    """q's output where k's input starts, or the reverse, would be written while other workgroups still read it."""
    far, odd = P + 0x200000, P + 1
    q, k = dict(x=P, y=P + 0x100000, w=odd), dict(x=far, y=far + 0x100000, w=odd)
    r = lambda a, b: _rope(lib, q=_heads(**{**q, **a}), k=_heads(**{**k, **b}))
    assert r({}, {}) == ERR_ALIGN                                  # apart: on to the alignment check
    assert r(dict(y=far), {}) == ERR_SHAPE and r({}, dict(y=P)) == ERR_SHAPE
    assert r(dict(y=far), dict(y=P)) == ERR_SHAPE                  # swapped
    assert r(dict(x=P, y=P), dict(x=P)) == ERR_SHAPE               # one input, q in place
    assert r(dict(x=P, y=P), dict(x=far, y=far)) == ERR_ALIGN      # both in place
    assert _rope(lib, q=_heads(**{**q, "y": far}), k=_heads(**{**k, "heads": 0})) == ERR_ALIGN  # no heads: not read
