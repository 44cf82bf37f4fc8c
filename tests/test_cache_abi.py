"""CPU tests of the paged cache's entry points: arguments are rejected before any launch (no GPU is touched), and the
binding's checks run before the library call."""

import ctypes
import os

import pytest

import w4a4_bit_quantized_amd as w4
from w4a4_bit_quantized_amd import binding

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED = 0, 1, 2, 3, 4
P = 0x10000  # a fake, well-aligned device address; never dereferenced by the validation paths
Q, OUT, K, V, WS = P, P + 0x1000000, P + 0x2000000, P + 0x3000000, P + 0x4000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        from w4a4_bit_quantized_amd import build
        build.build()
    return w4.load_library()


def cache(k=K, v=V, pages=8, page=16, heads=2, D=64, **kw):
    st = dict(kp=page * heads * D, kt=heads * D, kh=D, vp=page * heads * D, vt=heads * D, vh=D)
    st.update(kw)
    return binding.KvCache(k, v, pages, page, heads, st["kp"], st["kt"], st["kh"], st["vp"], st["vt"], st["vh"])


def side(x=P, ts=256, hs=64, heads=4, w=None, y=None, yts=256, yhs=64):
    return binding.Heads(x, ts, hs, heads, w, y, yts, yhs)


def append(lib, q=0, k=0, v=0, pos=P, T=4, D=64, dims=(64,), layout=0, flags=1, theta=1e4, eps=1e-6, dt=0, slots=P, c=0):
    q = side(y=OUT) if q == 0 else q
    k = side(x=P + 0x100000, heads=2) if k == 0 else k
    v = side(x=P + 0x200000, heads=2) if v == 0 else v
    c = cache() if c == 0 else c
    arr = (ctypes.c_int32 * max(len(dims), 1))(*dims)
    ref = lambda x: ctypes.byref(x) if x is not None else None
    return lib.w4a4_kv_append(ref(q), ref(k), ref(v), pos, T, D, len(dims), arr, layout, flags, theta, eps, dt, slots, ref(c),
                              None)


def test_append_validation(lib):
    r = lambda **kw: append(lib, **kw)
    assert r(dt=2) == ERR_UNSUPPORTED and r(dt=3) == ERR_UNSUPPORTED and r(layout=3) == ERR_UNSUPPORTED
    assert r(flags=16) == ERR_UNSUPPORTED and r(D=514) == ERR_UNSUPPORTED and r(dims=(2,) * 9) == ERR_UNSUPPORTED
    assert r(T=-1) == ERR_SHAPE and r(D=63) == ERR_SHAPE and r(dims=(66,)) == ERR_SHAPE and r(theta=0.0) == ERR_SHAPE
    assert r(k=None) == ERR_NULL and r(v=None) == ERR_NULL and r(c=None) == ERR_NULL
    assert r(c=cache(heads=3)) == ERR_SHAPE and r(v=side(heads=1)) == ERR_SHAPE
    assert r(c=cache(pages=-1)) == ERR_SHAPE and r(c=cache(page=0)) == ERR_SHAPE and r(c=cache(pages=1 << 31)) == ERR_SHAPE
    assert r(T=0, slots=None, pos=None, q=side(x=None)) == OK
    assert r(q=None, c=cache(pages=0, k=None, v=None)) == OK              # nothing to do
    assert r(slots=None) == ERR_NULL and r(pos=None) == ERR_NULL and r(c=cache(k=None)) == ERR_NULL
    assert r(q=side(x=None, y=OUT)) == ERR_NULL and r(q=side()) == ERR_NULL and r(k=side(x=None, heads=2)) == ERR_NULL
    assert r(slots=P + 2) == ERR_ALIGN and r(slots=P + 4, flags=9) == ERR_ALIGN and r(pos=P + 2) == ERR_ALIGN
    assert r(c=cache(v=V + 1)) == ERR_ALIGN and r(k=side(x=P + 0x100001, heads=2)) == ERR_ALIGN
    assert r(v=side(x=P + 0x200000, heads=2, w=P + 1), slots=P + 1) == ERR_ALIGN  # (v's weight is not read)


def test_append_places(lib):
    """Caches whose elements share an address, and outputs where inputs start, are refused."""
    odd = dict(slots=P + 1)                                               # accepted sizes reach the alignment check
    r = lambda **kw: append(lib, c=cache(**kw), **odd)
    assert r() == ERR_ALIGN
    assert r(kp=2 * 16 * 64, kh=16 * 64, kt=64) == ERR_ALIGN              # heads outside the page's tokens
    assert r(kt=8 * 2 * 64, kp=2 * 64) == ERR_ALIGN                       # pages inside tokens
    assert r(kh=8 * 16 * 64, kp=16 * 64, kt=64) == ERR_ALIGN              # heads outermost
    assert r(kh=63) == ERR_SHAPE and r(vt=127) == ERR_SHAPE and r(vp=16 * 128 - 1) == ERR_SHAPE and r(kt=0) == ERR_SHAPE
    assert r(pages=1, kp=0) == ERR_ALIGN and r(pages=1, page=1, kp=3, kt=5) == ERR_ALIGN
    assert r(kp=-1) == ERR_SHAPE and r(kp=1 << 41) == ERR_SHAPE and r(pages=1 << 22, kp=1 << 40) == ERR_SHAPE
    assert append(lib, c=cache(k=V), **odd) == ERR_SHAPE                  # both in one place
    assert append(lib, c=cache(k=P + 0x100000), **odd) == ERR_SHAPE       # on k's input
    assert append(lib, q=side(y=P + 0x100000), **odd) == ERR_SHAPE and append(lib, q=side(y=K), **odd) == ERR_SHAPE
    assert append(lib, q=side(y=P), **odd) == ERR_ALIGN                   # q in place


def attention(lib, c=0, ws=WS, wsb=1 << 40, tree=None, **kw):
    a = dict(q=Q, qt=256, qh=64, out=OUT, ot=256, oh=64, T=6, H=4, table=P, ts=8, tw=8, lens=P, starts=P, B=2, mq=3, window=0,
             sinks=0, scale=0.125, D=64, dt=0)
    a.update(kw)
    c = cache() if c == 0 else c
    s = binding.Attention(a["q"], a["qt"], a["qh"], a["out"], a["ot"], a["oh"], a["T"], a["H"], a["table"], a["ts"], a["tw"],
                          a["lens"], a["starts"], a["B"], a["mq"], a["window"], a["sinks"], a["scale"], a["D"], a["dt"])
    ref = (ctypes.byref(s), ctypes.byref(c) if c is not None else None)
    if tree is not None:
        return lib.w4a4_tree_attention(*ref, *tree, ws, wsb, None)
    return lib.w4a4_paged_attention(*ref, ws, wsb, None)


def test_attention_validation(lib):
    r = lambda **kw: attention(lib, **kw)
    assert r(dt=2) == ERR_UNSUPPORTED and r(dt=-1) == ERR_UNSUPPORTED and r(D=264) == ERR_UNSUPPORTED
    assert r(D=0) == ERR_SHAPE and r(D=60) == ERR_SHAPE and r(D=-8) == ERR_SHAPE
    assert r(T=-1) == ERR_SHAPE and r(B=-1) == ERR_SHAPE and r(H=0) == ERR_SHAPE and r(H=3) == ERR_SHAPE and r(c=cache(heads=0)) == ERR_SHAPE
    assert r(tw=-1) == ERR_SHAPE and r(window=-1) == ERR_SHAPE and r(sinks=-1) == ERR_SHAPE and r(mq=-1) == ERR_SHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert r(scale=scale) == ERR_SHAPE
    assert r(starts=None, T=7) == ERR_SHAPE                               # 7 queries of 2 sequences
    assert r(T=(1 << 28) + 1, qt=256, ot=256) == ERR_SHAPE                # tokens x heads past 2^30
    assert r(B=(1 << 30) + 1) == ERR_SHAPE and r(scale=3.4e38, lens=P + 1) == ERR_ALIGN
    assert r(T=0, q=None, out=None, lens=None, ws=None) == OK and r(B=0, T=0, lens=None) == OK
    for k in ("q", "out", "lens", "table"):
        assert r(**{k: None}) == ERR_NULL
    assert r(ws=None) == ERR_NULL and r(c=None) == ERR_NULL and r(c=cache(k=None)) == ERR_NULL
    assert r(out=Q) == ERR_SHAPE and r(out=K) == ERR_SHAPE and r(out=V) == ERR_SHAPE
    assert r(q=Q + 8) == ERR_ALIGN and r(out=OUT + 8) == ERR_ALIGN and r(c=cache(v=V + 8)) == ERR_ALIGN
    assert r(table=P + 2) == ERR_ALIGN and r(lens=P + 1) == ERR_ALIGN and r(starts=P + 2) == ERR_ALIGN and r(ws=WS + 128) == ERR_ALIGN
    assert r(c=cache(pages=0, k=None, v=None), table=None, lens=P + 1) == ERR_ALIGN  # no keys: the pool is not read


def test_attention_strides(lib):
    odd = dict(lens=P + 1)                                                # accepted sizes reach the alignment check
    r = lambda **kw: attention(lib, **{**odd, **kw})
    assert r() == ERR_ALIGN
    assert r(qt=252) == ERR_SHAPE and r(oh=68) == ERR_SHAPE and r(c=cache(kt=132)) == ERR_SHAPE and r(c=cache(vh=60)) == ERR_SHAPE
    assert r(ot=128) == ERR_SHAPE and r(oh=0) == ERR_SHAPE and r(ot=-256) == ERR_SHAPE and r(qt=1 << 41) == ERR_SHAPE
    assert r(qt=0, qh=0) == ERR_ALIGN                                     # broadcast queries
    assert r(ot=64, oh=6 * 64) == ERR_ALIGN                               # (heads, tokens, head_dim) output
    assert r(c=cache(kp=0, vp=0)) == ERR_ALIGN                            # all pages the same: they are only read
    assert r(H=1, qh=3, oh=5, c=cache(heads=1, kh=7)) == ERR_ALIGN        # one head: its stride does not matter
    assert r(c=cache(kp=1 << 31, vp=1 << 31)) == ERR_ALIGN and r(c=cache(kp=(1 << 31) + 8)) == ERR_SHAPE
    assert r(c=cache(vt=(1 << 31) + 8, vp=64)) == ERR_SHAPE and r(c=cache(kh=1 << 33)) == ERR_ALIGN
    assert r(c=cache(page=(1 << 31) - 1, kp=64, vp=64, kt=0, vt=0), tw=1 << 30) == ERR_ALIGN


def test_tree_validation(lib):
    r = lambda mask=P, ms=8, mw=3, pos=P, **kw: attention(lib, tree=(mask, ms, mw, pos), **kw)
    assert r(ms=-1) == ERR_SHAPE and r(mw=-1) == ERR_SHAPE and r(ms=1 << 41) == ERR_SHAPE
    assert r(mask=None) == ERR_NULL and r(pos=None, window=4) == ERR_NULL and r(mask=None, mw=0, lens=P + 1) == ERR_ALIGN
    assert r(pos=P + 2, window=4) == ERR_ALIGN and r(pos=None, lens=P + 1) == ERR_ALIGN


def test_workspace(lib):
    def need(T=6, B=2, H=4, heads=2, D=64, mq=3):
        a = binding.Attention(None, H * D, D, None, H * D, D, T, H, None, 0, 0, None, 1, B, mq, 0, 0, 1.0, D, 0)
        c = cache(heads=heads, D=D)
        return lib.w4a4_attention_workspace_bytes(ctypes.byref(a), ctypes.byref(c))
    n = need()
    if n == 0 and os.environ.get("W4A4_LIBRARY"):
        pytest.skip("a host-only build: no kernels, no workspace")
    assert n > 0 and n % 256 == 0 and need(D=60) == 0 and need(H=3) == 0
    assert attention(lib, wsb=n - 1) == ERR_SHAPE and attention(lib, wsb=n, lens=P + 1) == ERR_ALIGN
    # pieces of tiles: at least their rows' sums and outputs, of whole tiles of 128 rows in more slots than there are tiles
    for T, B, H, heads, D in ((506, 2, 16, 2, 128), (1012, 2, 16, 2, 128), (300, 7, 4, 4, 256), (65, 1, 64, 1, 64)):
        rows, wide = T * H // heads, 64 if D <= 64 else 128 if D <= 128 else 256
        pieces = min(16, max(1, 512 // (max(1, rows // 128) * heads)))
        assert pieces > 1
        assert need(T, B, H, heads, D, T) >= (rows // 128 + B) * heads * pieces * 128 * (2 + wide) * 4
    assert lib.w4a4_attention_workspace_bytes(None, None) == 0


def test_page_division():
    """The multiplier and shift that the kernels divide by: the largest remainders of every size that a page or a group may have."""
    import random
    rng = random.Random(1)
    sizes = list(range(1, 300)) + [2 ** k + d for k in range(9, 31) for d in (-1, 0, 1)] + [rng.randrange(1, 2 ** 31) for _ in range(200)]
    for d in sizes:
        shift = 31 + (d - 1).bit_length()
        mul = -(-(1 << shift) // d)
        assert mul < 1 << 32
        for x in [0, 1, d - 1, d, 2 ** 31 - 1] + [q * d + e for q in (1, (2 ** 31 - 1) // d - 1, rng.randrange(0, 2 ** 31 // d + 1)) for e in (-1, 0, d - 1)]:
            if 0 <= x < 2 ** 31:
                assert (x * mul) >> shift == x // d, (x, d)


def test_constants_match_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w4a4.h")).read()
    for name, value in (("W4A4_KV_SLOTS_I64", binding.KV_SLOTS_I64),
                        ("W4A4_ATTENTION_MAX_HEAD_DIM", binding.ATTENTION_MAX_HEAD_DIM)):
        assert f"#define {name} {value}\n" in text


def test_binding_refuses_host_tensors():
    import torch
    z = torch.zeros
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        w4.kv_append(None, z(4, 2, 64, **bf), z(4, 2, 64, **bf), z(4, dtype=torch.int32), [64], z(4, dtype=torch.int32),
                     z(2, 16, 2, 64, **bf), z(2, 16, 2, 64, **bf))
    with pytest.raises(ValueError, match="device tensor"):
        w4.paged_attention(z(4, 2, 64, **bf), z(2, 16, 2, 64, **bf), z(2, 16, 2, 64, **bf), z(4, 1, dtype=torch.int32),
                           z(4, dtype=torch.int32))
    with pytest.raises(TypeError, match="torch tensor"):
        w4.tree_attention(None, None, None, None, None, None)
