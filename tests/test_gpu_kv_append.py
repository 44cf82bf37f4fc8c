"""GPU parity of the append to a paged cache (needs an MI355X): q and k against ``oracle/rope.py`` with the tolerance
that tests/test_gpu_qk_norm_rope.py derives, v and everything that is not stored bit for bit."""

import numpy as np
import pytest

from test_gpu_qk_norm_rope import check, make, weights
from test_gpu_w8a8 import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a ROCm GPU"
    import w4a4_bit_quantized_amd as w
    w.load_library()
    return w


def drawn_slots(rng, T, pages, page, dropped):
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    for i, bad in zip(rng.permutation(T)[:dropped], (-1, pages * page, -2 ** 31, 2 ** 31 - 1) * dropped):
        slots[i] = bad
    return slots


def pool(rng, shape, dtype, order):
    """A (pages, page_size, heads, D) cache tensor whose memory is in another order."""
    import torch
    t = dev(make(rng, shape[0] * shape[1], shape[2], shape[3], dtype), dtype).view(*shape)
    if order == "heads_first":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if order == "wide":  # rows with a gap behind each head, pages with one behind them
        wide = torch.zeros(shape[0], shape[1] + 1, shape[2], shape[3] + 6, dtype=t.dtype, device=t.device)
        view = wide[:, :shape[1], :, :shape[3]]
        view.copy_(t)
        return view
    return t


SHAPES = [(1, 1, 1, 64, [64], 16), (1, 32, 8, 128, [128], 16), (5, 3, 1, 128, [16, 56, 56], 1), (130, 8, 8, 128, [44, 42, 42], 24),
          (600, 4, 2, 80, [16, 24, 24], 50), (2100, 5, 3, 64, [8, 24, 32], 64), (33, 2, 2, 256, [64, 64, 64, 64], 16),
          (9, 2, 1, 34, [2, 10, 6], 3), (17, 2, 3, 120, [40, 0, 48], 7), (2, 2, 1, 512, [510], 4), (70, 40, 2, 16, [8], 300)]


@pytest.mark.parametrize("layout", ["interleaved", "half", "axis_half"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(w4, shape, layout):
    import torch
    T, hq, hk, D, dims, page = shape
    for i, (dtype, order) in enumerate((("bf16", "plain"), ("f16", "heads_first"), ("bf16", "wide"))):
        print(f"\n{shape} {layout} {dtype} {order}", flush=True)
        rng = np.random.default_rng(i + T)
        pages, norm = T // page + 3, i != 2
        q, k, v = (make(rng, T, h, D, dtype) for h in (hq, hk, hk))
        qw, kw = (weights(rng, D, dtype), weights(rng, D, dtype)) if i else (None, None)
        pos = rng.integers(-1000, 1000, (T, len(dims)))
        slots = drawn_slots(rng, T, pages, page, T // 4)
        kc, vc = (pool(rng, (pages, page, hk, D), dtype, order) for _ in range(2))
        k0, v0 = host(kc.contiguous()).reshape(-1, hk, D), host(vc.contiguous()).reshape(-1, hk, D)
        yq = w4.kv_append(dev(q, dtype), dev(k, dtype), dev(v, dtype), torch.from_numpy(pos.astype(np.int32)).cuda(), dims,
                          torch.from_numpy(slots if i else slots.astype(np.int32)).cuda(), kc, vc,
                          None if qw is None else dev(qw, dtype), None if kw is None else dev(kw, dtype), layout=layout,
                          shared_frequencies=i == 1, norm=norm)
        torch.cuda.synchronize()
        check(yq, q, pos, dims, dtype, qw, layout, i == 1, norm, what="q")
        k1, v1 = host(kc.contiguous()).reshape(-1, hk, D), host(vc.contiguous()).reshape(-1, hk, D)
        kept = np.flatnonzero((slots >= 0) & (slots < pages * page))
        assert np.array_equal(v1[slots[kept]], v[kept])
        rest = np.setdiff1d(np.arange(pages * page), slots[kept])
        assert np.array_equal(v1[rest], v0[rest]) and np.array_equal(k1[rest], k0[rest])
        if kept.size:
            stored = torch.from_numpy(k1[slots[kept]].view(np.int16)).view(yq.dtype).cuda()
            check(stored, k[kept], pos[kept], dims, dtype, kw, layout, i == 1, norm, what="k")


def test_same_as_the_pass_without_a_cache(w4):
    """q's and k's results are qk_norm_rope's bit for bit, from partitions of a fused projection, q in place or not; gaps
    of a strided pool stay as they were."""
    import torch
    rng = np.random.default_rng(3)
    T, hq, hk, D, page = 70, 8, 2, 128, 16
    qkv = dev(make(rng, T, hq + 2 * hk, D, "bf16"), "bf16").view(T, -1)
    q, k, v = (x.view(T, -1, D) for x in qkv.split([hq * D, hk * D, hk * D], 1))
    pos = torch.arange(T, dtype=torch.int64, device="cuda") * 1000
    yq, yk = w4.qk_norm_rope(q, k, pos, [128], layout="half")
    slots = torch.randperm(8 * page, device="cuda")[:T]
    both = torch.zeros(8, 2, hk, page + 2, D + 8, dtype=torch.bfloat16, device="cuda")
    kc, vc = both[:, 0, :, :page, :D].transpose(1, 2), both[:, 1, :, :page, :D].transpose(1, 2)
    got = w4.kv_append(q, k, v, pos, [128], slots, kc, vc, layout="half")
    assert torch.equal(got, yq)
    kf, vf = kc.reshape(-1, hk, D), vc.reshape(-1, hk, D)
    assert torch.equal(kf[slots], yk) and torch.equal(vf[slots], v)
    assert both.count_nonzero() == kc.count_nonzero() + vc.count_nonzero()
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    assert w4.kv_append(None, k, v, pos, [128], slots, kc2, vc2, layout="half") is None
    assert torch.equal(kc2.reshape(-1, hk, D), kf) and torch.equal(vc2.reshape(-1, hk, D), vf)
    kept = qkv[:, hq * D:].clone()
    assert w4.kv_append(q, k, v, pos, [128], slots, kc2, vc2, layout="half", inplace=True) is q
    assert torch.equal(q, yq) and torch.equal(qkv[:, hq * D:], kept)
    empty = kc.new_empty(0, page, hk, D)
    assert torch.equal(w4.kv_append(yq, k, v, pos, [], slots, empty, empty.clone(), norm=False), yq)
