"""The measured cases of the paged key / value cache: appending to it, and attention over it.

``run`` computes each case either in plain elementary torch operations (``own`` false) or through
the package's entry points (``own`` true); ``exact`` gives the same outputs from the definitions
in 64 bits.

Append: each head of q and k goes through an RMS norm with a weight and a rotation of its pairs by
pos * frequency; q is returned, k and the unchanged v are stored at the token's slot (page * page
size + offset) of the cache; a token with a negative slot is not stored.

Attention: a sequence's n queries are the last n of its l keys, which lie in the pages that its row
of the page table names.  A query at position p sees keys j <= p with p - j < window or j < sinks.
Drafted tokens: the n queries are nodes of a tree at the cache's end; a node sees the keys before the
tree (within the window of its own position, or sinks) and those nodes that its row of the mask names.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decoded token's q, k and v: latency
        dict(name="append_token", op="append", T=1, hq=32, hk=8, D=128, page=16, pages=1024, axes="128", layout="half",
             shared=False, norm=True, weight=True, pad=0, x="bf16", far=100000),
        # a prompt of a model that rotates without a norm, from a fused projection's output
        dict(name="append_prompt", op="append", T=8192, hq=32, hk=8, D=128, page=64, pages=160, axes="128", layout="half",
             shared=False, norm=False, weight=False, pad=0, x="bf16", far=32768),
        # part of the head rotated by three axes, odd pages, a batch padded to its graph's size
        dict(name="append_ragged", op="append", T=1237, hq=14, hk=2, D=80, page=24, pages=70, axes="16,24,24",
             layout="interleaved", shared=True, norm=True, weight=True, pad=37, x="f16", far=20000),
        # one decoded token of one sequence: latency
        dict(name="decode_token", op="attend", B=1, n0=1, n1=1, l0=4096, l1=4096, hq=32, hk=8, D=128, page=16, window=0,
             sinks=0, x="bf16"),
        # a batch of decoded tokens, from sequences just begun to long ones: bandwidth
        dict(name="decode_batch", op="attend", B=64, n0=1, n1=1, l0=37, l1=8191, hq=32, hk=8, D=128, page=16, window=0,
             sinks=0, x="bf16"),
        # long streams in a layer with a sliding window and kept first tokens
        dict(name="decode_window", op="attend", B=16, n0=1, n1=1, l0=30000, l1=32768, hq=32, hk=4, D=128, page=64,
             window=4096, sinks=4, x="f16"),
        # a long prompt, all of it at once: the largest product
        dict(name="prompt", op="attend", B=1, n0=8192, n1=8192, l0=8192, l1=8192, hq=32, hk=8, D=128, page=64, window=0,
             sinks=0, x="bf16"),
        # several prompts of odd lengths in a layer with a sliding window
        dict(name="prompt_window", op="attend", B=4, n0=1000, n1=4001, l0=1000, l1=4001, hq=16, hk=4, D=64, page=32,
             window=1024, sinks=4, x="f16"),
        # the next piece of two prompts that are taken in pieces
        dict(name="prompt_piece", op="attend", B=2, n0=500, n1=512, l0=12000, l1=16384, hq=16, hk=2, D=128, page=128,
             window=0, sinks=0, x="bf16"),
        # one sequence's drafted tokens: latency
        dict(name="tree_token", op="tree", B=1, n0=16, n1=16, l0=2000, l1=2000, hq=32, hk=8, D=128, page=16, window=0,
             sinks=0, x="bf16"),
        # a batch of trees of different sizes over contexts of different lengths
        dict(name="tree_batch", op="tree", B=16, n0=33, n1=64, l0=1000, l1=8192, hq=32, hk=8, D=128, page=16, window=0,
             sinks=0, x="bf16"),
        # small trees in a layer with a sliding window, odd heads and pages
        dict(name="tree_window", op="tree", B=5, n0=7, n1=27, l0=500, l1=5000, hq=14, hk=2, D=80, page=24, window=1024,
             sinks=8, x="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "tree"])
    D = rng.choice([64, 128, 128, 128, 256, 72, 80, 96, 120])
    hk = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hk * rng.choice([1, 2, 4, 4, 5, 7, 8])
    while hq * D > 8192:
        hq, hk = hk, hk if hq > hk else hk // 2
        hk = min(hk, hq)
    page = rng.choice([16, 16, 32, 64, 128, 256, 1, 24, 50])
    x = rng.choice(["bf16", "bf16", "f16"])
    if op == "append":
        T = _log(rng, 1, 8192)
        while T * (hq + 2 * hk) * D > 8192 * 48 * 128:
            T = max(1, T // 2)
        n = rng.choice([1, 1, 2, 3])
        rot = D if rng.random() < 0.6 else 2 * rng.randint(n, D // 2)
        cuts = sorted(rng.sample(range(1, rot // 2), n - 1)) if n > 1 else []
        dims = [2 * (b - a) for a, b in zip([0] + cuts, cuts + [rot // 2])]
        return dict(op=op, T=T, hq=hq, hk=hk, D=D, page=page, pages=T // page + rng.randint(1, 40),
                    axes=",".join(str(d) for d in dims), layout=rng.choice(["interleaved", "half", "axis_half"]),
                    shared=rng.random() < 0.3, norm=rng.random() < 0.6, weight=rng.random() < 0.7,
                    pad=rng.choice([0, 0, T // 9]), x=x, far=_log(rng, 8, 1000000))
    window = rng.choice([0, 0, _log(rng, 16, 8192)])
    sinks = rng.choice([0, 4, rng.randint(1, 100)]) if window else 0
    kind = "tree" if op == "tree" else rng.choice(["decode", "decode", "prompt", "piece"])
    while True:
        if kind == "decode":
            B, n1, l1 = _log(rng, 1, 128), 1, _log(rng, 1, 65536)
        elif kind == "tree":
            B, n1, l1 = _log(rng, 1, 32), rng.randint(2, 64), _log(rng, 64, 32768)
        elif kind == "prompt":
            B, l1 = _log(rng, 1, 16), _log(rng, 16, 8192)
            n1 = l1
        else:
            B, n1, l1 = rng.randint(1, 4), _log(rng, 2, 1024), _log(rng, 2048, 32768)
        # no more keys and pairs than the largest listed cases have
        if B * l1 * hk * D <= 64 * 4096 * 8 * 128 and B * n1 * hq * l1 * D <= 8192 * 8192 * 32 * 128 // 2:
            break
    n0 = n1 if kind == "decode" else rng.randint(max(1, n1 // 3), n1)
    l0 = n0 if kind == "prompt" else max(n1, rng.randint(max(1, l1 // 8), l1))
    if B == 1:
        n0, l0 = n1, l1
    return dict(op=op, B=B, n0=n0, n1=n1, l0=l0, l1=l1, hq=hq, hk=hk, D=D, page=page, window=window, sinks=sinks, x=x)


def _spread(lo, hi, n):
    """n whole numbers from lo to hi."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _batch(case):
    """(queries, keys) of every sequence, before they are put into an order."""
    return list(zip(_spread(case["n0"], case["n1"], case["B"]), _spread(case["l0"], case["l1"], case["B"])))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    dev, dt = "cuda", DT[case["x"]]
    hq, hk, D, page = case["hq"], case["hk"], case["D"], case["page"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    s = dict(case=case)
    if case["op"] == "append":
        T, pages = case["T"], case["pages"]
        # a fused projection's output holds the q, k and v partitions side by side in each row
        qkv = (normal(T, (hq + 2 * hk) * D) * 1.5).to(dt)
        s["q"] = qkv[:, :hq * D].view(T, hq, D)
        s["k"] = qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
        s["v"] = qkv[:, (hq + hk) * D:].view(T, hk, D)
        s["qw"] = (1 + 0.2 * normal(D)).to(dt) if case["weight"] else None
        s["kw"] = (1 + 0.2 * normal(D)).to(dt) if case["weight"] else None
        s["dims"] = [int(d) for d in case["axes"].split(",")]
        s["pos"] = torch.randint(0, case["far"], (T, len(s["dims"])), generator=g, device=dev, dtype=torch.int32)
        # the tokens fill pages in the order in which a pool hands them out
        order = torch.randperm(pages, generator=g, device=dev)
        t = torch.arange(T, device=dev)
        s["slots"] = order[t // page] * page + t % page
        s["slots"][T - case["pad"]:] = -1
        s["kc"], s["vc"] = normal(pages, page, hk, D).to(dt), normal(pages, page, hk, D).to(dt)
        return s
    B = case["B"]
    both = _batch(case)
    both = [both[i] for i in torch.randperm(B, generator=host).tolist()]
    ns, ls = [n for n, _ in both], [l for _, l in both]
    need = [(l + page - 1) // page for l in ls]
    pages = sum(need) + 8
    # every sequence's pages lie anywhere in the pool; the table's unused entries name none
    order = torch.randperm(pages, generator=host).to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    starts = [0]
    for n in ns:
        starts.append(starts[-1] + n)
    T = starts[-1]
    s["table"], s["lens"] = table.to(dev), torch.tensor(ls, dtype=torch.int32, device=dev)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["max_q"] = max(ns)
    s["kc"], s["vc"] = normal(pages, page, hk, D).to(dt), normal(pages, page, hk, D).to(dt)
    s["q"] = (normal(T, hq, D) * 1.5).to(dt)
    if case["op"] == "tree":
        mask = torch.zeros(T, max(ns), dtype=torch.bool)
        pos = torch.zeros(T, dtype=torch.int32)
        for b in range(B):
            for i in range(ns[b]):
                r = starts[b] + i
                # node i hangs under an earlier node, mostly a recent one; node 0 is the last accepted token
                if i:
                    back = int(torch.randint(1, min(i, 8) + 1, (1,), generator=host))
                    mask[r] = mask[r - back]
                    pos[r] = pos[r - back] + 1
                else:
                    pos[r] = ls[b] - ns[b]
                mask[r, i] = True
        s["mask"], s["pos"] = mask.to(dev), pos.to(dev)
    return s


def _pairs(case, dims, pos):
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


def _plain_heads(x, norm, w, i0, i1, cos, sin):
    u = x.float()
    if norm:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-6)
        if w is not None:
            u = u * w.float()
    y = u.clone()
    a, b = u[..., i0], u[..., i1]
    y[..., i0] = a * cos[:, None] - b * sin[:, None]
    y[..., i1] = a * sin[:, None] + b * cos[:, None]
    return y.to(x.dtype)


def _plain_append(s):
    case = s["case"]
    i0, i1, ang = _pairs(case, s["dims"], s["pos"])
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    q = _plain_heads(s["q"], case["norm"], s["qw"], i0, i1, cos, sin)
    k = _plain_heads(s["k"], case["norm"], s["kw"], i0, i1, cos, sin)
    stored = case["T"] - case["pad"]  # the padded tokens are the last ones
    slots = s["slots"][:stored]
    s["kc"].view(-1, case["hk"], case["D"])[slots] = k[:stored]
    s["vc"].view(-1, case["hk"], case["D"])[slots] = s["v"][:stored]
    return q, s["kc"], s["vc"]


def _plain_attention(s):
    """All sequences at once, padded to the longest."""
    case = s["case"]
    hq, hk, D, page = case["hq"], case["hk"], case["D"], case["page"]
    starts, lens, B, N, L = s["starts"].long(), s["lens"].long(), case["B"], case["n1"], case["l1"]
    n = starts[1:] - starts[:-1]
    i, j = torch.arange(N, device="cuda"), torch.arange(L, device="cuda")
    rows = torch.minimum(starts[:-1, None] + i, starts[1:, None] - 1)               # (B, N) rows of q, the last one repeated
    jj = torch.minimum(j, lens[:, None] - 1)                                        # (B, L) keys, the last one repeated
    slots = torch.gather(s["table"].long(), 1, jj // page) * page + jj % page
    q = s["q"][rows].float().view(B, N, hk, hq // hk, D).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, D)
    k = s["kc"].view(-1, hk, D)[slots].float().permute(0, 2, 1, 3).contiguous()     # (B, hk, L, D)
    v = s["vc"].view(-1, hk, D)[slots].float().permute(0, 2, 1, 3).contiguous()
    before = (lens - n)[:, None, None]                                              # keys before the queries
    if case["op"] == "tree":
        p = s["pos"][rows].long()[:, :, None]
        node = torch.clamp(j - before, 0, N - 1).expand(B, N, L)
        tree = torch.gather(s["mask"][rows], 2, node) & (j - before < n[:, None, None])
        inside = j < before
    else:
        p = before + i[:, None]
        tree = torch.zeros((), dtype=torch.bool, device="cuda")
        inside = (j <= p) & (j < lens[:, None, None])
    if case["window"]:
        inside = inside & ((p - j < case["window"]) | (j < case["sinks"]))
    seen = torch.where(j < before, inside, inside | tree)                           # (B, N, L)
    sc = (q @ k.transpose(-1, -2)).view(B, hk, N, hq // hk, L) * (1.0 / math.sqrt(D))
    sc = sc.masked_fill(~seen[:, None, :, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    sc = torch.exp(sc - torch.where(top == -math.inf, 0.0, top))
    total = sc.sum(-1, keepdim=True)
    o = (sc.view(B, hk, -1, L) @ v).view(B, hk, N, hq // hk, D) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, N, hq, D)
    return o[i < n[:, None]].to(s["q"].dtype)


def run(state):
    case = state["case"]
    if own:
        import w4a4_bit_quantized_amd as w4
        if case["op"] == "append":
            q = w4.kv_append(state["q"], state["k"], state["v"], state["pos"], state["dims"], state["slots"], state["kc"],
                             state["vc"], q_weight=state["qw"], k_weight=state["kw"], eps=1e-6, theta=10000.0,
                             layout=case["layout"], shared_frequencies=case["shared"], norm=case["norm"])
            return q, state["kc"], state["vc"]
        if case["op"] == "tree":
            return w4.tree_attention(state["q"], state["kc"], state["vc"], state["table"], state["lens"], state["mask"],
                                     q_starts=state["starts"], max_q=state["max_q"], positions=state["pos"],
                                     window=case["window"], sinks=case["sinks"])
        return w4.paged_attention(state["q"], state["kc"], state["vc"], state["table"], state["lens"],
                                  q_starts=state["starts"], max_q=state["max_q"], window=case["window"],
                                  sinks=case["sinks"])
    return _plain_append(state) if case["op"] == "append" else _plain_attention(state)


def _seen(case, n, l):
    """(pairs of a query and a key that it sees, keys that any query sees) of one sequence; a tree's nodes
    are taken as a chain, which has the most pairs."""
    window, sinks = case["window"], case["sinks"]
    pairs = 0
    for p in range(l - n, l):
        pairs += min(p + 1, window + min(sinks, max(0, p + 1 - window))) if window else p + 1
    first = max(0, l - n + 1 - window) if window else 0
    return pairs, l - first + min(sinks, first)


def work(case):
    hq, hk, D = case["hq"], case["hk"], case["D"]
    if case["op"] == "append":
        T, stored = case["T"], case["T"] - case["pad"]
        # read q, k and v, write q and what is stored; positions and slots
        n = T * hq + stored * hk
        return {"bytes": 2 * D * (2 * n + 2 * stored * hk) + T * (4 * len(case["axes"].split(",")) + 8), "flops": 8 * n * D}
    rows = pairs = keys = 0
    for n, l in _batch(case):
        a, b = _seen(case, n, l)
        rows, pairs, keys = rows + n, pairs + a, keys + b
    mask = rows * case["n1"] + 4 * rows if case["op"] == "tree" else 0
    return {"bytes": 4 * rows * hq * D + 4 * keys * hk * D + 4 * (keys // case["page"] + 3 * case["B"]) + mask,
            "flops": 4 * pairs * hq * D}


def _exact_append(case, s):
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
        if case["norm"]:
            d = d / torch.sqrt(d.pow(2).sum(-1, keepdim=True) / d.shape[-1] + 1e-6)
            if w is not None:
                d = d * w.to(torch.float64)
        r = torch.complex(d[..., lo], d[..., hi]) * z
        d[..., lo], d[..., hi] = r.real, r.imag
        outs.append(d)
    q, k = outs
    kc, vc = s["kc"].to(torch.float64), s["vc"].to(torch.float64)
    kept = s["slots"] >= 0
    page, off = s["slots"][kept] // case["page"], s["slots"][kept] % case["page"]
    kc[page, off] = k[kept]
    vc[page, off] = s["v"].to(torch.float64)[kept]
    return q, kc, vc


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    hq, hk, D = case["hq"], case["hk"], case["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for b, l in enumerate(lens):
        first, n = starts[b], starts[b + 1] - starts[b]
        pages = s["table"][b, :(l + case["page"] - 1) // case["page"]].long()
        keys = s["kc"][pages].reshape(-1, hk, D)[:l].to(torch.float64)
        vals = s["vc"][pages].reshape(-1, hk, D)[:l].to(torch.float64)
        j = torch.arange(l, device="cuda")
        for at in range(0, n, 1024):  # queries in pieces: the scores of all would not fit
            i = torch.arange(at, min(n, at + 1024), device="cuda")
            place = s["pos"][first + i].long() if case["op"] == "tree" else i + (l - n)
            gap = place[:, None] - j
            ok = torch.ones_like(gap, dtype=torch.bool) if case["op"] == "tree" else gap >= 0
            if case["window"]:
                ok = ok & ((gap < case["window"]) | (j < case["sinks"])[None])
            if case["op"] == "tree":
                ok[:, l - n:] = s["mask"][first + i][:, :n]
            for h in range(hq):
                w = torch.matmul(s["q"][first + i, h].to(torch.float64), keys[:, h * hk // hq].t().contiguous()) / math.sqrt(D)
                w = torch.softmax(w.masked_fill(~ok, -math.inf), -1)
                out[first + i, h] = torch.matmul(torch.nan_to_num(w), vals[:, h * hk // hq].contiguous())
    return out
