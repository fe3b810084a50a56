"""The operators of a layer whose checkpoint routes by scores and keeps its weights in 8-bit floating point, with their
plain forms: routing by softmax or sigmoid scores with a balance bias, groups and scaled weights (moe_router_scored),
E4M3 codes with a scale per block of 128 (moe_fp8_quant), the product of activations with such weights
(moe_fp8_matmul) and the routed experts' SwiGLU feed-forward on them (moe_fp8_expert_ffn_combine).

listed() and draw() give cases, prepare() a case's inputs, run() one pass (the library's kernels where `own` is
true, plain torch operations otherwise), exact() the same outputs in 64 bits, work() what a pass cannot do without.
"""
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3 = torch.float8_e4m3fn
TOP = 448.0  # the largest E4M3 value
TINY = 2.0 ** -126  # the smallest scale

# the largest listed cases: what a drawn case may cost at most
MOST_ROUTE = 2048 * 6144 * 256
MOST_ROUTERS = 16 * 256 * 6144
MOST_QUANT = 2048 * 6144
MOST_MACS = 2048 * 6144 * 6144
MOST_WEIGHTS = 65536 * 4096
MOST_EXPERTS = 128 * 4096 * 1536
MOST_EXPERT_MACS = 2048 * 9 * 4096 * 1536


def listed():
    return [
        # one new token's routing by sigmoid scores with a balance bias: launch latency
        {"name": "route token", "op": "route", "layers": 1, "T": 1, "H": 4096, "E": 128, "k": 8, "score": "sigmoid",
         "balance": True, "groups": 1, "top": 1, "rule": "max", "renorm": True, "scale": 1.0},
        # the routers of every layer of a batched decode step in one call, softmax over all experts, best groups
        {"name": "route step", "op": "route", "layers": 16, "T": 32, "H": 6144, "E": 256, "k": 8, "score": "softmax",
         "balance": False, "groups": 8, "top": 3, "rule": "max", "renorm": False, "scale": 16.0},
        # a prompt chunk: sigmoid, balance bias, the groups of the two largest sums
        {"name": "route prompt", "op": "route", "layers": 1, "T": 2048, "H": 6144, "E": 256, "k": 8,
         "score": "sigmoid", "balance": True, "groups": 8, "top": 4, "rule": "top2", "renorm": True, "scale": 2.5},
        # a prompt chunk's hidden states on their way into a product
        {"name": "quant prompt", "op": "quant", "type": "bf16", "rows": 2048, "K": 6144, "block": 1, "rule": "amax"},
        # a checkpoint's matrix in blocks of 128 x 128, the last ones cut short in both directions
        {"name": "quant weights", "op": "quant", "type": "fp32", "rows": 1533, "K": 2080, "block": 128,
         "rule": "pow2"},
        # a projection of one token in decode
        {"name": "matmul token", "op": "matmul", "M": 1, "N": 4096, "K": 4096, "out": "bf16", "bias": False},
        # a projection of a batched decode step
        {"name": "matmul batch", "op": "matmul", "M": 32, "N": 6144, "K": 6144, "out": "bf16", "bias": False},
        # odd sizes in every direction, with a bias, fp32 out
        {"name": "matmul ragged", "op": "matmul", "M": 333, "N": 1001, "K": 1568, "out": "fp32", "bias": True},
        # a prompt chunk's projection
        {"name": "matmul prompt", "op": "matmul", "M": 2048, "N": 6144, "K": 6144, "out": "bf16", "bias": False},
        # the experts of one token in decode, and the shared one
        {"name": "experts token", "op": "experts", "T": 1, "H": 4096, "I": 1536, "E": 128, "k": 8, "shared": True},
        # a batched decode step: most experts have a token or two
        {"name": "experts batch", "op": "experts", "T": 32, "H": 4096, "I": 1536, "E": 128, "k": 8, "shared": False},
        # a prompt chunk: about a hundred tokens an expert
        {"name": "experts prompt", "op": "experts", "T": 2048, "H": 4096, "I": 1536, "E": 128, "k": 8,
         "shared": True},
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "quant", "matmul", "matmul", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _log(rng, 2, 64)
        E, top = groups * size, rng.randint(1, groups)
        k = rng.randint(1, min(12, top * size))
        H = 32 * _log(rng, 2, 192)
        layers = rng.choice([1, 1, 1, 3, 8])
        T = _log(rng, 1, max(1, min(2048, MOST_ROUTE // (layers * E * H))))
        return {"op": op, "layers": layers, "T": T, "H": H, "E": E, "k": k,
                "score": rng.choice(["softmax", "sigmoid"]), "balance": rng.random() < 0.5, "groups": groups,
                "top": top, "rule": rng.choice(["max", "top2"]), "renorm": rng.random() < 0.5,
                "scale": rng.choice([1.0, 2.5, 16.0])}
    if op == "quant":
        K = 16 * _log(rng, 1, 384)
        rows = _log(rng, 1, min(8192, MOST_QUANT // K))
        return {"op": op, "type": rng.choice(["bf16", "fp16", "fp32"]), "rows": rows, "K": K,
                "block": rng.choice([1, 128]), "rule": rng.choice(["amax", "pow2"])}
    if op == "matmul":
        K = 16 * _log(rng, 4, 384)
        M = _log(rng, 1, 2048)
        N = _log(rng, 16, min(65536, MOST_WEIGHTS // K, MOST_MACS // (K * M)))
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "fp32"]), "bias": rng.random() < 0.5}
    H, I = 32 * _log(rng, 2, 128), 32 * _log(rng, 2, 64)
    E = _log(rng, 4, min(256, MOST_EXPERTS // (H * I)))
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, max(1, min(2048, MOST_EXPERT_MACS // ((k + 1) * H * I))))
    return {"op": op, "T": T, "H": H, "I": I, "E": E, "k": k, "shared": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _blocks(n):
    return (n + 127) // 128


def _hidden(rows, width, gen, dtype):
    """Hidden states: N(0,1) with a few channels much larger than the others, as trained networks have them."""
    x = torch.randn((rows, width), generator=gen, device=DEV)
    big = torch.rand((width,), generator=gen, device=DEV) < 0.004
    return (x * torch.where(big, 24.0, 1.0)).to(dtype)


def _weights(rows, width, gen):
    """(codes, scales) of a matrix N(0, 0.02^2) in blocks of 128 x 128."""
    codes, scales = _quantise(torch.randn((rows, width), generator=gen, device=DEV) * 0.02, 128, "amax")
    return codes.view(torch.uint8), scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        Lyr, T, H, E, k = case["layers"], case["T"], case["H"], case["E"], case["k"]
        s["x"] = _hidden(Lyr * T, H, gen, torch.bfloat16).view(Lyr, T, H)
        s["w"] = torch.randn((Lyr, E, H), generator=gen, device=DEV) * (1.0 / H ** 0.5)
        s["b"] = torch.randn((Lyr, E), generator=gen, device=DEV) * 0.05 if case["balance"] else None
        s["idx"] = torch.empty((Lyr, T, k), dtype=torch.int32, device=DEV)
        s["wt"] = torch.empty((Lyr, T, k), dtype=torch.float32, device=DEV)
    elif case["op"] == "quant":
        R, K, dt = case["rows"], case["K"], TYPES[case["type"]]
        if case["block"] == 1:
            s["x"] = _hidden(R, K, gen, dt)
        else:  # weights: each row with a size of its own
            size = 0.02 * torch.exp(0.5 * torch.randn((R, 1), generator=gen, device=DEV))
            s["x"] = (torch.randn((R, K), generator=gen, device=DEV) * size).to(dt)
        s["stride"] = (_blocks(K) + 3) // 4 * 4
        s["codes"] = torch.empty((R, K), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((R if case["block"] == 1 else _blocks(R), s["stride"]), device=DEV)
    elif case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _hidden(M, K, gen, torch.bfloat16)
        s["w"], s["ws"] = _weights(N, K, gen)
        s["b"] = torch.randn((N,), generator=gen, device=DEV) if case["bias"] else None
        s["y"] = torch.empty((M, N), dtype=TYPES[case["out"]], device=DEV)
    else:
        T, H, I, E, k = case["T"], case["H"], case["I"], case["E"], case["k"]
        s["x"] = _hidden(T, H, gen, torch.bfloat16)
        # an expert's slab: W1 [I,H], W3 [I,H] and W2 [H,I] codes, then their scales, then zeros to 16 bytes
        n = E + (1 if case["shared"] else 0)
        scales = 2 * _blocks(I) * _blocks(H) + _blocks(H) * _blocks(I)
        s["slabs"] = torch.zeros((n, (3 * H * I + 4 * scales + 15) // 16 * 16), dtype=torch.uint8, device=DEV)
        for e in range(n):
            parts = [_weights(*shape, gen) for shape in ((I, H), (I, H), (H, I))]
            at = 0
            for part in [p[0] for p in parts] + [p[1].view(torch.uint8) for p in parts]:
                s["slabs"][e, at:at + part.numel()] = part.reshape(-1)
                at += part.numel()
        s["table"] = s["slabs"].data_ptr() + s["slabs"].shape[1] * torch.arange(E, device=DEV, dtype=torch.int64)
        # each token's experts, without repeats, and weights that sum to one
        s["idx"] = torch.rand((T, E), generator=gen, device=DEV).argsort(dim=1)[:, :k].int().contiguous()
        s["wt"] = torch.softmax(torch.randn((T, k), generator=gen, device=DEV), dim=1)
        s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _pow2(e):
    """2^e in 64 bits, exactly, for whole e in -1022..1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _spread(scales, block_rows, rows, K):
    """A scale per element from a scale per block."""
    return scales.repeat_interleave(block_rows, dim=0)[:rows].repeat_interleave(128, dim=1)[:, :K]


def _quantise(x, block_rows, rule):
    """(E4M3 codes, scales in 32 bits) of x's blocks of block_rows x 128: the scale puts the largest magnitude at 448
    (amax), or is the smallest power of two that leaves it at most there (pow2); 1 for a block of zeros."""
    rows, K = x.shape
    R, C = -(-rows // block_rows), _blocks(K)
    full = torch.zeros((R * block_rows, C * 128), device=x.device)
    full[:rows, :K] = x.float().abs()
    top = full.view(R, block_rows, C, 128).amax(dim=(1, 3)).double()
    if rule == "pow2":
        m, e = torch.frexp(top / TOP)  # m in [0.5, 1)
        scales = _pow2(torch.where(m == 0.5, e - 1, e))
    else:
        scales = top / TOP
    scales = torch.where(top > 0, scales.clamp(min=TINY), 1.0).float()
    q = x.double() / _spread(scales, block_rows, rows, K).double()
    _, e = torch.frexp(q)
    step = _pow2(torch.clamp(e - 1, min=-6) - 3)  # four significant bits, and 2^-9 below 2^-6
    q = (torch.round(q / step) * step).clamp(-TOP, TOP)
    return q.float().to(E4M3), scales


def _values(codes, scales, block_rows):
    """The values that E4M3 codes and their scales stand for, in 32 bits."""
    rows, K = codes.shape
    return codes.view(E4M3).float() * _spread(scales, block_rows, rows, K)


def _plain_route(s):
    Lyr, T, E, k = s["layers"], s["T"], s["E"], s["k"]
    logits = (s["x"].double() @ s["w"].double().transpose(1, 2)).float().double()  # one rounding to 32 bits
    p = torch.softmax(logits, dim=-1) if s["score"] == "softmax" else torch.sigmoid(logits)
    c = p if s["b"] is None else p + s["b"].double().unsqueeze(1)
    if s["groups"] > 1:
        g = c.view(Lyr, T, s["groups"], -1)
        best = g.sort(dim=-1, descending=True)[0]
        of = best[..., 0] if s["rule"] == "max" else best[..., :2].sum(-1)
        keep = of.sort(dim=-1, descending=True, stable=True)[1][..., :s["top"]]
        inside = torch.zeros_like(of, dtype=torch.bool).scatter_(-1, keep, True)
        c = torch.where(inside.unsqueeze(-1), g, -float("inf")).view(Lyr, T, E)
    idx = c.sort(dim=-1, descending=True, stable=True)[1][..., :k]
    w = p.gather(-1, idx)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"idx": idx.int(), "w": (s["scale"] * w).float()}


def _matrices(s, e):
    """An expert's matrices, from its slab, in 32 bits."""
    H, I = s["H"], s["I"]
    shapes = ((I, H), (I, H), (H, I))
    slab, at, codes, mats = s["slabs"][e], 0, [], []
    for r, c in shapes:
        codes.append(slab[at:at + r * c].view(r, c))
        at += r * c
    for (r, c), m in zip(shapes, codes):
        n = 4 * _blocks(r) * _blocks(c)
        mats.append(_values(m, slab[at:at + n].view(torch.float32).view(_blocks(r), _blocks(c)), 128))
        at += n
    return mats


def _feed_forward(x, mats):
    """The down projection of an expert's quantised SwiGLU of quantised rows."""
    g, u = x @ mats[0].t(), x @ mats[1].t()
    return _values(*_quantise(g * torch.sigmoid(g) * u, 1, "amax"), 1) @ mats[2].t()


def _plain(s):
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "quant":
        codes, scales = _quantise(s["x"], s["block"], s["rule"])
        return {"codes": codes, "scales": scales}
    x = _values(*_quantise(s["x"], 1, "amax"), 1)
    if s["op"] == "matmul":
        y = x @ _values(s["w"], s["ws"], 128).t()
        if s["b"] is not None:
            y = y + s["b"]
        return {"y": y.to(TYPES[s["out"]])}
    T, k = s["T"], s["k"]
    y = torch.zeros((T * k, s["H"]), device=DEV)  # row t * k + i: token t's expert i
    for e in torch.unique(s["idx"]).tolist():
        pairs = (s["idx"].reshape(-1) == e).nonzero().squeeze(1)
        y[pairs] = _feed_forward(x[pairs // k], _matrices(s, e))
    out = (y.view(T, k, -1) * s["wt"].unsqueeze(-1)).sum(1)
    if s["shared"]:
        out = out + _feed_forward(x, _matrices(s, s["E"]))
    return {"out": out.to(torch.bfloat16)}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    from routed_expert_streaming_amd import _lib as L
    stream = torch.cuda.current_stream()
    types = {"bf16": L.MOE_BF16, "fp16": L.MOE_FP16, "fp32": L.MOE_FP32}
    if s["op"] == "route":
        Lyr, T, H, E, k = s["layers"], s["T"], s["H"], s["E"], s["k"]
        if "how" not in s:  # the description and the workspace that a program keeps
            s["how"] = L.moe_routing(L.MOE_SCORE_SOFTMAX if s["score"] == "softmax" else L.MOE_SCORE_SIGMOID,
                                     s["groups"], s["top"],
                                     L.MOE_GROUP_MAX if s["rule"] == "max" else L.MOE_GROUP_TOP2,
                                     int(s["renorm"]), s["scale"])
            s["space"] = L.moe_router_scored_workspace_bytes(Lyr, T, E, H)
            s["work"] = torch.empty(s["space"], dtype=torch.uint8, device=DEV)
        L.moe_router_scored(s["x"], Lyr, T, H, s["w"], None, s["b"], E, k, s["how"], s["idx"], s["wt"], s["work"],
                            s["space"], stream)
        return {"idx": s["idx"], "w": s["wt"]}
    if s["op"] == "quant":
        K = s["K"]
        L.moe_fp8_quant(s["x"], types[s["type"]], K * SIZE[s["type"]], s["rows"], K, s["block"],
                        L.MOE_FP8_SCALE_POW2 if s["rule"] == "pow2" else L.MOE_FP8_SCALE_AMAX, s["codes"], K,
                        s["scales"], 4 * s["stride"], stream)
        return {"codes": s["codes"].view(E4M3), "scales": s["scales"][:, :_blocks(K)]}
    if s["op"] == "matmul":
        M, N, K = s["M"], s["N"], s["K"]
        if "space" not in s:
            s["space"] = L.moe_fp8_matmul_workspace_bytes(M, N, K, L.MOE_BF16)
            s["work"] = torch.empty(max(s["space"], 1), dtype=torch.uint8, device=DEV)
        # bf16 activations are quantised on the way in
        L.moe_fp8_matmul(s["x"], L.MOE_BF16, 2 * K, None, 0, s["w"], K, s["ws"], 4 * _blocks(K), M, N, K, s["b"],
                         s["y"], types[s["out"]], N * SIZE[s["out"]], s["work"], s["space"], stream)
        return {"y": s["y"]}
    T, H, I, E, k = s["T"], s["H"], s["I"], s["E"], s["k"]
    if "space" not in s:
        s["space"] = L.moe_fp8_expert_ffn_workspace_bytes(T, H, I, E, k, s["shared"])
        s["work"] = torch.empty(s["space"], dtype=torch.uint8, device=DEV)
    L.moe_fp8_expert_ffn_combine(s["x"], T, H, I, E, s["idx"], s["wt"], k, s["table"],
                                 s["slabs"][E] if s["shared"] else None, s["out"], s["work"], s["space"], stream)
    return {"out": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _grid():
    """The 127 magnitudes of E4M3 in the order of their codes."""
    code = torch.arange(127, device=DEV, dtype=torch.float64)
    e, m = torch.floor(code / 8), code % 8
    return torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e - 7))


def _nearest(x, block_rows, rule):
    """(code values, scales) of x in 64 bits: each value the nearest of the magnitudes, ties to the even code."""
    rows, K = x.shape
    x = x.double()
    code, scales = torch.empty_like(x), torch.empty((-(-rows // block_rows), _blocks(K)), dtype=torch.float64,
                                                    device=x.device)
    grid = _grid()
    middle = (grid[1:] + grid[:-1]) / 2
    for j in range(_blocks(K)):
        part = x[:, 128 * j:128 * j + 128]
        top = part.abs().amax(dim=1)
        if block_rows > 1:
            whole = torch.nn.functional.pad(top, (0, -rows % block_rows))
            top = whole.view(-1, block_rows).amax(dim=1)
        s = top / TOP
        if rule == "pow2":
            e = torch.ceil(torch.log2(torch.where(top > 0, s, 1.0)))
            e = torch.where(torch.exp2(e) < s, e + 1, e)  # log2 may round across a whole number
            e = torch.where(torch.exp2(e - 1) >= s, e - 1, e)
            s = torch.exp2(e)
        # the scale is kept in 32 bits, and what the codes are is for that scale
        s = torch.where(top > 0, s.clamp(min=TINY), 1.0).float().double()
        scales[:, j] = s
        u = part.abs() / s.repeat_interleave(block_rows)[:rows].unsqueeze(1)
        i = torch.bucketize(u, middle)  # ties: the lower of the two
        tie = u == middle[i.clamp(max=125)]
        i = torch.where(tie & (i < 126) & (i % 2 == 1), i + 1, i)
        code[:, 128 * j:128 * j + 128] = torch.copysign(grid[i], part)
    return code, scales


def _wide(codes, scales, block_rows):
    """Values in 64 bits, from code values and scales."""
    rows, K = codes.shape
    r = torch.arange(rows, device=codes.device) // block_rows
    c = torch.arange(K, device=codes.device) // 128
    return codes.double() * scales.double()[r][:, c]


def _bytes_wide(codes):
    """The values of E4M3 bytes, in 64 bits."""
    b = codes.long()
    return _grid()[(b & 127).clamp(max=126)] * torch.where(b > 127, -1.0, 1.0)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "route":
        Lyr, T, E, k = s["layers"], s["T"], s["E"], s["k"]
        idx = torch.empty((Lyr, T, k), dtype=torch.int32, device=DEV)
        w = torch.empty((Lyr, T, k), dtype=torch.float64, device=DEV)
        n = E // s["groups"]
        for l in range(Lyr):
            # the router's logits are defined as rounded once to 32 bits
            logit = (s["w"][l].double() @ s["x"][l].double().t()).t().float().double()
            if s["score"] == "softmax":
                p = torch.exp(logit - logit.amax(1, keepdim=True))
                p = p / p.sum(1, keepdim=True)
            else:
                p = 1 / (1 + torch.exp(-logit))
            c = p.clone() if s["b"] is None else p + s["b"][l].double()
            if s["groups"] > 1:
                worth = torch.empty((T, s["groups"]), dtype=torch.float64, device=DEV)
                for g in range(s["groups"]):
                    best = torch.topk(c[:, g * n:g * n + n], min(2, n), dim=1)[0]
                    worth[:, g] = best[:, 0] if s["rule"] == "max" else best.sum(1)
                for _ in range(s["groups"] - s["top"]):  # drop the least one, the last of equals
                    low = s["groups"] - 1 - worth.flip(1).argmin(1)
                    worth.scatter_(1, low[:, None], float("inf"))
                out = worth == float("inf")
                c = c.masked_fill(out.repeat_interleave(n, dim=1), -float("inf"))
            for i in range(k):  # the largest one left, the first of equals
                top = c.amax(1, keepdim=True)
                first = (c == top).int().argmax(1, keepdim=True)
                idx[l, :, i] = first[:, 0].int()
                w[l, :, i] = p.gather(1, first)[:, 0]
                c.scatter_(1, first, -float("inf"))
        if s["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        return {"idx": idx, "w": w * s["scale"]}
    if s["op"] == "quant":
        codes, scales = _nearest(s["x"], s["block"], s["rule"])
        return {"codes": codes, "scales": scales}
    x = _wide(*_nearest(s["x"], 1, "amax"), 1)
    if s["op"] == "matmul":
        y = torch.empty((s["M"], s["N"]), dtype=torch.float64, device=DEV)
        for n in range(0, s["N"], 8192):
            w = _wide(_bytes_wide(s["w"][n:n + 8192]), s["ws"][n // 128:n // 128 + 64], 128)
            y[:, n:n + 8192] = x @ w.t()
        if s["b"] is not None:
            y += s["b"].double()
        return {"y": y}
    T, H, I, k = s["T"], s["H"], s["I"], s["k"]
    hb, ib = _blocks(H), _blocks(I)

    def expert(e, rows):
        slab = s["slabs"][e]
        f = slab[3 * H * I:3 * H * I + 12 * hb * ib].view(torch.float32)
        w1 = _wide(_bytes_wide(slab[:H * I].view(I, H)), f[:hb * ib].view(ib, hb), 128)
        w3 = _wide(_bytes_wide(slab[H * I:2 * H * I].view(I, H)), f[hb * ib:2 * hb * ib].view(ib, hb), 128)
        w2 = _wide(_bytes_wide(slab[2 * H * I:3 * H * I].view(H, I)), f[2 * hb * ib:].view(hb, ib), 128)
        g = rows @ w1.t()
        h = g / (1 + torch.exp(-g)) * (rows @ w3.t())
        return _wide(*_nearest(h, 1, "amax"), 1) @ w2.t()

    out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for e in range(s["E"]):
        t, i = (s["idx"] == e).nonzero(as_tuple=True)
        if len(t):
            out.index_add_(0, t, expert(e, x[t]) * s["wt"][t, i].double().unsqueeze(1))
    if s["shared"]:
        out += expert(s["E"], x)
    return {"out": out}


def work(case):
    if case["op"] == "route":
        Lyr, T, H, E, k = case["layers"], case["T"], case["H"], case["E"], case["k"]
        return {"bytes": Lyr * (2 * T * H + 4 * E * H + (4 * E if case["balance"] else 0) + 8 * T * k),
                "flops": 2 * Lyr * T * H * E}
    if case["op"] == "quant":  # the input, the codes and the scales
        R, K = case["rows"], case["K"]
        return {"bytes": R * K * (SIZE[case["type"]] + 1) + 4 * -(-R // case["block"]) * _blocks(K), "flops": 4 * R * K}
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K + 4 * _blocks(N) * _blocks(K) + M * N * SIZE[case["out"]]
                + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    T, H, I, E, k = case["T"], case["H"], case["I"], case["E"], case["k"]
    used = E * (1 - (1 - k / E) ** T) + case["shared"]  # experts that some token picks, on average
    return {"bytes": used * (3 * H * I + 12 * _blocks(H) * _blocks(I)) + 4 * T * H + 8 * T * k,
            "flops": 6 * H * I * T * (k + case["shared"])}
