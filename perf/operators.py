"""The measured cases of the W8A8 linear layer and of the q / k head norm with rotary positions.

``run`` computes each case either in plain elementary torch operations (``own`` false) or through
the package's entry points (``own`` true); ``exact`` gives the same outputs from the definitions
in 64 bits.

W8A8 layer: v = x / smooth_factor (optionally rotated per block by H / sqrt(B)); per token
a = amax|v| / 127 and q = round(v * 127 / amax); y = (q @ qweight^T) * a * wscales + bias.

q / k: per head an RMS norm with a weight, then a rotation of pairs by pos * frequency, the pairs
divided among the position axes.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token through a projection: latency
        dict(name="linear_token", op="linear", M=1, K=2048, N=6144, block=0, bias=False, x="bf16", y="bf16"),
        # the framework's small-batch workload (16 rows, weight streaming) in 8 bits
        dict(name="linear_batch16", op="linear", M=16, K=5120, N=13824, block=0, bias=True, x="bf16", y="bf16"),
        # a batch of decoded tokens, rotated input, the output in f16
        dict(name="linear_batch48_rot", op="linear", M=48, K=4096, N=4096, block=64, bias=False, x="f16", y="f16"),
        # a short prompt with odd sizes: K ends inside a K step, N inside a tile and off 16-byte rows
        dict(name="linear_ragged", op="linear", M=301, K=1552, N=4099, block=16, bias=True, x="bf16", y="bf16"),
        # attention output projection of an image's tokens
        dict(name="linear_proj", op="linear", M=4096, K=2048, N=2048, block=0, bias=True, x="bf16", y="bf16"),
        # MLP up-projection of a prompt or an image: the largest product
        dict(name="linear_up", op="linear", M=4096, K=5120, N=13824, block=0, bias=True, x="bf16", y="bf16"),
        # rotated MLP down-projection (the framework's rotated K = 12288 workload): large quantizer share
        dict(name="linear_down_rot", op="linear", M=4096, K=12288, N=2560, block=128, bias=False, x="bf16", y="bf16"),
        # one quantized activation multiplied again (a second projection of the same input), f32 out
        dict(name="gemm_shared", op="gemm", M=1021, K=4096, N=2050, bias=True, y="f32"),
        # one decoded token: latency
        dict(name="rope_token", op="rope", T=1, hq=32, hk=8, D=128, axes="128", layout="half", shared=False,
             fused=True, weight=True, x="bf16", far=100000),
        # text and image tokens of a fused QKV projection's output, three axes
        dict(name="rope_image", op="rope", T=4608, hq=24, hk=24, D=128, axes="16,56,56", layout="interleaved",
             shared=False, fused=True, weight=True, x="bf16", far=128),
        # video tokens, three axes, the largest
        dict(name="rope_video", op="rope", T=32760, hq=24, hk=24, D=128, axes="44,42,42", layout="interleaved",
             shared=False, fused=False, weight=True, x="bf16", far=1024),
        # grouped heads, part of the head rotated, one frequency ladder over three sections, f32, odd counts
        dict(name="rope_ragged", op="rope", T=1237, hq=14, hk=2, D=80, axes="16,24,24", layout="half", shared=True,
             fused=True, weight=True, x="f32", far=20000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "gemm", "rope", "rope"])
    if kind != "rope":
        while True:
            M, K, N = _log(rng, 1, 4096), 16 * _log(rng, 4, 768), _log(rng, 32, 13824)
            if M * K * N <= 4096 * 5120 * 13824:
                break
        y = rng.choice(["bf16", "f16"])
        if kind == "gemm":
            return dict(op="gemm", M=M, K=K, N=N, bias=rng.random() < 0.5, y=rng.choice([y, "f32"]))
        blocks = [b for b in (0, 0, 16, 32, 64, 128) if b == 0 or K % b == 0]
        return dict(op="linear", M=M, K=K, N=N, block=rng.choice(blocks), bias=rng.random() < 0.5,
                    x=rng.choice(["bf16", "bf16", "f16", "f32"]), y=y)
    D = rng.choice([64, 64, 128, 128, 128, 256, 72, 80, 96, 120, 34])
    T, hk = _log(rng, 1, 32760), rng.choice([1, 2, 3, 4, 8, 12, 24])
    hq = hk * rng.choice([1, 1, 2, 4, 5])
    while T * (hq + hk) * D > 32760 * 48 * 128:
        T = max(1, T // 2)
    n = rng.choice([1, 2, 3, 3, 4])
    rot = D if rng.random() < 0.6 else 2 * rng.randint(n, D // 2)
    cuts = sorted(rng.sample(range(1, rot // 2), n - 1)) if n > 1 else []
    dims = [2 * (b - a) for a, b in zip([0] + cuts, cuts + [rot // 2])]
    return dict(op="rope", T=T, hq=hq, hk=hk, D=D, axes=",".join(str(d) for d in dims),
                layout=rng.choice(["interleaved", "half", "axis_half"]), shared=rng.random() < 0.3,
                fused=rng.random() < 0.6, weight=rng.random() < 0.8, x=rng.choice(["bf16", "bf16", "f16", "f32"]),
                far=_log(rng, 8, 1000000))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device=dev, dtype=torch.float32) * (hi - lo) + lo

    s = dict(case=case)
    if case["op"] == "rope":
        T, hq, hk, D, dt = case["T"], case["hq"], case["hk"], case["D"], DT[case["x"]]
        # a fused projection's output holds q, k and v partitions side by side in each row
        if case["fused"]:
            qkv = (normal(T, (hq + 2 * hk) * D) * 1.5).to(dt)
            s["q"] = qkv[:, :hq * D].view(T, hq, D)
            s["k"] = qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
        else:
            s["q"] = (normal(T, hq, D) * 1.5).to(dt)
            s["k"] = (normal(T, hk, D) * 1.5).to(dt)
        s["qw"] = uniform(0.5, 1.5, D).to(dt) if case["weight"] else None
        s["kw"] = uniform(0.5, 1.5, D).to(dt) if case["weight"] else None
        dims = [int(d) for d in case["axes"].split(",")]
        s["pos"] = torch.randint(0, case["far"], (T, len(dims)), generator=g, device=dev, dtype=torch.int32)
        s["dims"] = dims
        return s
    M, K, N = case["M"], case["K"], case["N"]
    # weights as an offline quantizer leaves them: one scale per output channel, N(0, 1/K)
    w = normal(N, K) / math.sqrt(K)
    ws = w.abs().amax(1) / 127.0
    s["layer"] = dict(qweight=torch.round(w / ws[:, None]).clamp_(-127, 127).to(torch.int8), wscales=ws)
    del w
    if case["bias"]:
        s["layer"]["bias"] = uniform(-1, 1, N).to(torch.bfloat16)
    # tokens with a few outlier channels, as the framework's synthetic workloads draw them
    x = normal(M, K)
    out = torch.randperm(K, generator=g, device=dev)[:max(1, K // 100)]
    x[:, out] *= 20.0
    if case["op"] == "gemm":
        a = x.abs().amax(1) / 127.0
        s["qact"], s["ascales"] = torch.round(x / a[:, None]).clamp_(-127, 127).to(torch.int8), a
    else:
        s["x"] = x.to(DT[case["x"]])
        s["layer"]["smooth_factor"] = uniform(0.5, 2.0, K).to(torch.bfloat16)
    return s


def _sylvester(B, dtype):
    """H_B with entries (-1)^popcount(i & j)."""
    i = torch.arange(B, device="cuda")
    b = i[:, None] & i[None, :]
    odd = (b ^ (b >> 1) ^ (b >> 2) ^ (b >> 3) ^ (b >> 4) ^ (b >> 5) ^ (b >> 6)) & 1
    return (1 - 2 * odd).to(dtype)


def _pairs(case, dims, T, pos):
    """Element indices (i0, i1) of every rotated pair, and the pairs' angles (T, rot / 2) in 64 bits."""
    rot = sum(dims)
    half = torch.tensor(dims, device="cuda") // 2
    axis = torch.repeat_interleave(torch.arange(len(dims), device="cuda"), half, output_size=rot // 2)
    p = torch.arange(rot // 2, device="cuda")
    first = (torch.cumsum(half, 0) - half)[axis]  # the first pair of the pair's axis
    i = p - first
    if case["layout"] == "interleaved":
        i0, i1 = 2 * p, 2 * p + 1
    elif case["layout"] == "half":
        i0, i1 = p, p + rot // 2
    else:
        i0 = 2 * first + i
        i1 = i0 + half[axis]
    e = p.double() / (rot // 2) if case["shared"] else i.double() / half[axis].double()
    return i0, i1, pos.double()[:, axis] * torch.pow(10000.0, -e)


def _plain_heads(x, w, i0, i1, cos, sin):
    u = x.float()
    u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-6)
    if w is not None:
        u = u * w.float()
    y = u.clone()
    a, b = u[..., i0], u[..., i1]
    y[..., i0] = a * cos[:, None] - b * sin[:, None]
    y[..., i1] = a * sin[:, None] + b * cos[:, None]
    return y.to(x.dtype)


def run(state):
    case = state["case"]
    if own:
        import w4a4_bit_quantized_amd as w4
        if case["op"] == "rope":
            return w4.qk_norm_rope(state["q"], state["k"], state["pos"], state["dims"], q_weight=state["qw"],
                                   k_weight=state["kw"], eps=1e-6, theta=10000.0, layout=case["layout"],
                                   shared_frequencies=case["shared"])
        layer = state["layer"]
        if case["op"] == "gemm":
            return w4.w8a8_gemm(state["qact"], state["ascales"], layer["qweight"], layer["wscales"],
                                bias=layer.get("bias"), out_dtype=DT[case["y"]])
        return w4.w8a8_linear(state["x"], layer, hadamard_block=case["block"], out_dtype=DT[case["y"]])
    if case["op"] == "rope":
        i0, i1, ang = _pairs(case, state["dims"], case["T"], state["pos"])
        cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
        return (_plain_heads(state["q"], state["qw"], i0, i1, cos, sin),
                _plain_heads(state["k"], state["kw"], i0, i1, cos, sin))
    layer = state["layer"]
    if case["op"] == "gemm":
        q, a = state["qact"].float(), state["ascales"]
    else:
        v = state["x"].float() / layer["smooth_factor"].float()
        B = case["block"]
        if B:
            v = ((v.view(-1, B) @ _sylvester(B, torch.float32)) * (1.0 / math.sqrt(B))).view(v.shape)
        amax = v.abs().amax(1)
        a = amax / 127.0
        q = torch.round(v * (127.0 / amax)[:, None])
    y = (q @ layer["qweight"].float().t()) * a[:, None] * layer["wscales"]
    if case["bias"]:
        y = y + layer["bias"].float()
    return y.to(DT[case["y"]])


def work(case):
    es = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "rope":
        n = case["T"] * (case["hq"] + case["hk"]) * case["D"]
        axes = len(case["axes"].split(","))
        # read and write every element, read the positions; square and sum, scale, rotate
        return {"bytes": 2 * n * es[case["x"]] + 4 * case["T"] * axes, "flops": 8 * n}
    M, K, N = case["M"], case["K"], case["N"]
    x = M * K + 4 * M if case["op"] == "gemm" else M * K * es[case["x"]] + 2 * K
    return {"bytes": x + N * K + 4 * N + (2 * N if case["bias"] else 0) + M * N * es[case["y"]],
            "flops": 2 * M * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        dims, rot = s["dims"], sum(s["dims"])
        freq, lo, hi, ax = [], [], [], []
        for a, d in enumerate(dims):
            base = sum(dims[:a])
            for j in range(d // 2):
                p = base // 2 + j
                freq.append(10000.0 ** (-2.0 * p / rot) if case["shared"] else 10000.0 ** (-2.0 * j / d))
                ax.append(a)
                i0, i1 = {"interleaved": (2 * p, 2 * p + 1), "half": (p, p + rot // 2),
                          "axis_half": (base + j, base + j + d // 2)}[case["layout"]]
                lo.append(i0)
                hi.append(i1)
        lo, hi = torch.tensor(lo, device="cuda"), torch.tensor(hi, device="cuda")
        turn = s["pos"].to(torch.float64)[:, torch.tensor(ax, device="cuda")]
        turn = turn * torch.tensor(freq, dtype=torch.float64, device="cuda")
        z = torch.polar(torch.ones_like(turn), turn)[:, None, :]
        outs = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            d = x.to(torch.float64)
            d = d / torch.sqrt(d.pow(2).sum(-1, keepdim=True) / d.shape[-1] + 1e-6)
            if w is not None:
                d = d * w.to(torch.float64)
            r = torch.complex(d[..., lo], d[..., hi]) * z
            d[..., lo], d[..., hi] = r.real, r.imag
            outs.append(d)
        return tuple(outs)
    w = s["layer"]["qweight"].to(torch.float64)
    if case["op"] == "gemm":
        codes, scale = s["qact"].to(torch.float64), s["ascales"].to(torch.float64)
    else:
        v = s["x"].to(torch.float64) / s["layer"]["smooth_factor"].to(torch.float64)
        if case["block"]:
            h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
            while h.shape[0] < case["block"]:
                h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
            v = torch.matmul(v.reshape(-1, case["block"]), h).reshape(v.shape) / math.sqrt(case["block"])
        top = v.abs().max(dim=1).values
        scale = top / 127
        codes = torch.round(v / scale[:, None])
    y = torch.matmul(codes, w.t().contiguous()) * scale[:, None] * s["layer"]["wscales"].to(torch.float64)
    if case["bias"]:
        y = y + s["layer"]["bias"].to(torch.float64)
    return y
