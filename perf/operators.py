"""The dense operators around the routed experts, with their plain forms: MXFP4 quantisation of rows
(moe_mx_quant), the product of activations with MXFP4 weight rows (moe_mx_matmul) and the norms before and after a
block with its gate and residual scale (moe_block_norm).

listed() and draw() give cases, prepare() a case's inputs, run() one pass (the library's kernels where `own` is
true, plain torch operations otherwise), exact() the same outputs in 64 bits, work() what a pass cannot do without.
"""
import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the codes 0..7; codes 8..15 are their negatives
EPS = 1e-6

# the largest listed cases: what a drawn case may cost at most
MOST_QUANT = 2048 * 6144
MOST_MACS = 2048 * 6144 * 6144
MOST_WEIGHTS = 65536 * 4096
MOST_NORM = 2048 * 6144


def row_bytes(K):
    """Bytes of an MXFP4 row: K/2 of codes, K/32 of scales, padded to 16."""
    return (K // 2 + K // 32 + 15) // 16 * 16


def listed():
    return [
        # one new token's hidden state on its way into an MXFP4 product: launch latency
        {"name": "quant token", "op": "quant", "type": "bf16", "rows": 1, "K": 4096, "rule": "floor"},
        # a 2048-token prompt chunk's hidden states
        {"name": "quant prompt", "op": "quant", "type": "bf16", "rows": 2048, "K": 6144, "rule": "floor"},
        # a checkpoint's weight matrix made into MXFP4, odd row count, last 128-column group cut short
        {"name": "quant weights", "op": "quant", "type": "fp32", "rows": 1533, "K": 2080, "rule": "fit"},
        # a dense projection of one token in decode, activations kept in bf16
        {"name": "matmul token", "op": "matmul", "act": "bf16", "M": 1, "N": 4096, "K": 4096, "out": "bf16",
         "bias": False},
        # logits of four sequences over a vocabulary: the longest weight stream
        {"name": "matmul logits", "op": "matmul", "act": "bf16", "M": 4, "N": 65536, "K": 4096, "out": "fp32",
         "bias": False},
        # a batched decode step's projection, activations quantised on the way in
        {"name": "matmul batch", "op": "matmul", "act": "mx", "M": 32, "N": 6144, "K": 6144, "out": "bf16",
         "bias": False},
        # odd sizes in every direction, with a bias, fp32 out
        {"name": "matmul ragged", "op": "matmul", "act": "mx", "M": 333, "N": 1001, "K": 1568, "out": "fp32",
         "bias": True},
        # a prompt chunk's projection, both operands in 4 bits
        {"name": "matmul prompt", "op": "matmul", "act": "mx", "M": 2048, "N": 6144, "K": 6144, "out": "bf16",
         "bias": False},
        # the same chunk with bf16 activations
        {"name": "matmul prompt bf16", "op": "matmul", "act": "bf16", "M": 2048, "N": 4096, "K": 6144, "out": "bf16",
         "bias": True},
        # one token between two blocks, post-norm and pre-norm weights
        {"name": "norm token", "op": "norm", "T": 1, "H": 4096, "resid": "fp32", "post": True, "gate": "none"},
        # a prompt chunk between two blocks, learned per-channel gate
        {"name": "norm prompt", "op": "norm", "T": 2048, "H": 6144, "resid": "fp32", "post": True,
         "gate": "channel"},
        # odd width, residual stream in bf16, a gate value per element
        {"name": "norm ragged", "op": "norm", "T": 301, "H": 1001, "resid": "bf16", "post": True, "gate": "element"},
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["quant", "matmul", "matmul", "norm"])
    if op == "quant":
        K = 32 * _log(rng, 1, 192)
        rows = _log(rng, 1, min(8192, MOST_QUANT // K))
        return {"op": op, "type": rng.choice(["bf16", "fp16", "fp32"]), "rows": rows, "K": K,
                "rule": rng.choice(["floor", "fit"])}
    if op == "matmul":
        K = 32 * _log(rng, 2, 192)
        M = _log(rng, 1, 2048)
        N = _log(rng, 16, min(65536, MOST_WEIGHTS // K, MOST_MACS // (K * M)))
        return {"op": op, "act": rng.choice(["bf16", "mx"]), "M": M, "N": N, "K": K,
                "out": rng.choice(["bf16", "fp32"]), "bias": rng.random() < 0.5}
    H = _log(rng, 32, 6144)
    T = _log(rng, 1, min(8192, MOST_NORM // H))
    return {"op": op, "T": T, "H": H, "resid": rng.choice(["fp32", "bf16"]), "post": rng.random() < 0.7,
            "gate": rng.choice(["none", "channel", "row", "element"])}


# ------------------------------------------------------------------ inputs
def _hidden(rows, width, gen, dtype):
    """Hidden states: N(0,1) with a few channels much larger than the others, as trained networks have them."""
    x = torch.randn((rows, width), generator=gen, device=DEV)
    big = torch.rand((width,), generator=gen, device=DEV) < 0.004
    return (x * torch.where(big, 24.0, 1.0)).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    if case["op"] == "quant":
        R, K, dt = case["rows"], case["K"], TYPES[case["type"]]
        if case["type"] == "bf16":
            s["x"] = _hidden(R, K, gen, dt)
        else:  # weights: each row with a size of its own
            size = 0.02 * torch.exp(0.5 * torch.randn((R, 1), generator=gen, device=DEV))
            s["x"] = (torch.randn((R, K), generator=gen, device=DEV) * size).to(dt)
        s["rows_out"] = torch.empty((R, row_bytes(K)), dtype=torch.uint8, device=DEV)
        s["values"] = torch.empty((R, K), dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _hidden(M, K, gen, torch.bfloat16)
        s["w"] = _pack(torch.randn((N, K), generator=gen, device=DEV) * 0.02)
        s["b"] = torch.randn((N,), generator=gen, device=DEV) if case["bias"] else None
        s["xq"] = torch.empty((M, row_bytes(K)), dtype=torch.uint8, device=DEV)  # the quantised activations
        s["y"] = torch.empty((M, N), dtype=TYPES[case["out"]], device=DEV)
    else:
        T, H = case["T"], case["H"]
        s["add"] = _hidden(T, H, gen, torch.bfloat16)
        s["r"] = (4 * _hidden(T, H, gen, torch.float32)).to(TYPES[case["resid"]])
        s["w_post"] = 1 + 0.2 * torch.randn((H,), generator=gen, device=DEV)
        s["w_pre"] = 1 + 0.2 * torch.randn((H,), generator=gen, device=DEV)
        shape = {"none": None, "channel": (H,), "row": (T,), "element": (T, H)}[case["gate"]]
        g = None if shape is None else torch.rand(shape, generator=gen, device=DEV)
        s["g"] = g.to(torch.bfloat16) if case["gate"] == "element" else g
        s["scale"] = 0.22
        s["r_out"] = torch.empty_like(s["r"])
        s["x_next"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _pow2(e):
    """2^e in 32 bits, exactly, for whole e in -127..127 (int32 tensors)."""
    return ((e.clamp(min=-126) + 127) << 23).view(torch.float32) * torch.where(e < -126, 0.5, 1.0)


def _quantise(x, rule):
    """(codes, scale exponents, values) of x's blocks of 32: the shared exponent from the block's largest magnitude,
    the elements to the nearest E2M1 magnitude, ties to the even code, larger ones to 6."""
    xb = x.float().reshape(x.shape[0], -1, 32)
    top = xb.abs().amax(-1, keepdim=True)
    bits = top.view(torch.int32)
    e = (bits >> 23) - 127 - 2
    if rule == "fit":  # no element beyond 6 * 2^e
        e = e + ((bits & 0x7FFFFF) > 0x400000).int()
    e = e.clamp(-127, 127)
    m = xb.abs() * _pow2(-e)
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int()
            + (m >= 3.5).int() + (m > 5.0).int())
    neg = torch.signbit(xb)
    values = torch.tensor(E2M1, device=x.device)[code] * _pow2(e)
    values = torch.where(neg, -values, values).reshape(x.shape)
    return (code + 8 * neg.int()).reshape(x.shape), e.squeeze(-1), values


def _pack(w):
    """MXFP4 rows (codes, then scale bytes, then zeros to a multiple of 16) of w, [rows, K] in 32 bits."""
    codes, e, _ = _quantise(w, "floor")
    rows = torch.zeros((w.shape[0], row_bytes(w.shape[1])), dtype=torch.uint8, device=w.device)
    K = w.shape[1]
    rows[:, :K // 2] = (codes[:, 0::2] + 16 * codes[:, 1::2]).to(torch.uint8)
    rows[:, K // 2:K // 2 + K // 32] = (e + 127).to(torch.uint8)
    return rows


def _unpack(rows, K):
    """The values of MXFP4 rows, in 32 bits."""
    b = rows[:, :K // 2].int()
    codes = torch.stack([b & 15, b >> 4], dim=-1).reshape(rows.shape[0], K // 32, 32)
    signed = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)
    scale = _pow2(rows[:, K // 2:K // 2 + K // 32].int() - 127)
    return (signed[codes] * scale.unsqueeze(-1)).reshape(rows.shape[0], K)


def _rms(v, w):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * w


def _plain(s):
    if s["op"] == "quant":
        return {"values": _quantise(s["x"], s["rule"])[2].to(torch.bfloat16)}
    if s["op"] == "matmul":
        x = _quantise(s["x"], "floor")[2] if s["act"] == "mx" else s["x"].float()
        y = x @ _unpack(s["w"], s["K"]).t()
        if s["b"] is not None:
            y = y + s["b"]
        return {"y": y.to(TYPES[s["out"]])}
    d = s["add"].float()
    if s["post"]:
        d = _rms(d, s["w_post"])
    if s["gate"] != "none":
        g = s["g"].float()
        d = d * (g.unsqueeze(-1) if s["gate"] == "row" else g)
    r = (s["r"].float() + s["scale"] * d).to(TYPES[s["resid"]])
    return {"resid": r, "x_next": _rms(r.float(), s["w_pre"]).to(torch.bfloat16)}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    from routed_expert_streaming_amd import _lib as L
    stream = torch.cuda.current_stream()
    types = {"bf16": L.MOE_BF16, "fp16": L.MOE_FP16, "fp32": L.MOE_FP32}
    if s["op"] == "quant":
        K = s["K"]
        rule = L.MOE_MX_SCALE_FIT if s["rule"] == "fit" else L.MOE_MX_SCALE_FLOOR
        L.moe_mx_quant(s["x"], types[s["type"]], K * SIZE[s["type"]], s["rows"], K, rule, s["rows_out"],
                       row_bytes(K), s["values"], stream)
        return {"values": s["values"]}
    if s["op"] == "matmul":
        M, N, K = s["M"], s["N"], s["K"]
        a, a_type, a_stride = s["x"], L.MOE_BF16, 2 * K
        if s["act"] == "mx":
            L.moe_mx_quant(a, L.MOE_BF16, 2 * K, M, K, L.MOE_MX_SCALE_FLOOR, s["xq"], row_bytes(K), None, stream)
            a, a_type, a_stride = s["xq"], L.MOE_MXFP4, row_bytes(K)
        if "ws" not in s:  # a workspace that a program keeps
            s["ws_bytes"] = L.moe_mx_matmul_workspace_bytes(M, N, K, a_type)
            s["ws"] = torch.empty(max(s["ws_bytes"], 1), dtype=torch.uint8, device=DEV)
        L.moe_mx_matmul(a, a_type, a_stride, s["w"], row_bytes(K), M, N, K, s["b"], s["y"], types[s["out"]],
                        N * SIZE[s["out"]], s["ws"], s["ws_bytes"], stream)
        return {"y": s["y"]}
    gates = {"none": L.MOE_GATE_NONE, "channel": L.MOE_GATE_CHANNEL, "row": L.MOE_GATE_ROW,
             "element": L.MOE_GATE_ELEMENT}
    L.moe_block_norm(s["add"], s["post"], s["w_post"] if s["post"] else None, s["g"], gates[s["gate"]], s["scale"],
                     s["r"], s["r_out"], types[s["resid"]], s["w_pre"], s["T"], s["H"], EPS, s["x_next"], None,
                     stream)
    return {"resid": s["r_out"], "x_next": s["x_next"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _nearest(x, rule):
    """MXFP4 values of x in 64 bits, each the nearest of the eight magnitudes by distance."""
    v = x.double().reshape(-1, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e = torch.where(torch.exp2(e) > top, e - 1, e)  # log2 may round across a whole number
    e = torch.where(torch.exp2(e + 1) <= top, e + 1, e) - 2
    if rule == "fit":
        e = torch.where(top > 6 * torch.exp2(e), e + 1, e)
    e = torch.where(top > 0, e, -127.0).clamp(-127, 127)
    u = v.abs() / torch.exp2(e)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    best, off = torch.zeros_like(u), u.clone()  # the distance to 0
    for j in (2, 4, 6, 1, 3, 5, 7):  # even codes first: an odd one has to be nearer
        d = (u - grid[j]).abs()
        near = d < off
        best, off = torch.where(near, grid[j], best), torch.where(near, d, off)
    return (torch.copysign(best, v) * torch.exp2(e)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quant":
        return {"values": _nearest(s["x"], s["rule"])}
    if s["op"] == "matmul":
        K = s["K"]
        x = _nearest(s["x"], "floor") if s["act"] == "mx" else s["x"].double()
        byte = torch.arange(16, device=DEV)
        mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[byte % 8] * torch.where(byte > 7, -1.0, 1.0)
        y = torch.zeros((s["M"], s["N"]), dtype=torch.float64, device=DEV)
        for n in range(0, s["N"], 8192):
            w = torch.empty((min(8192, s["N"] - n), K), dtype=torch.float64, device=DEV)
            codes = s["w"][n:n + 8192, :K // 2].long()
            w[:, 0::2], w[:, 1::2] = mag[codes % 16], mag[codes // 16]
            scale = torch.exp2(s["w"][n:n + 8192, K // 2:K // 2 + K // 32].double() - 127)
            y[:, n:n + 8192] = x @ (w * scale.repeat_interleave(32, dim=1)).t()
        if s["b"] is not None:
            y += s["b"].double()
        return {"y": y}
    d = s["add"].double()
    if s["post"]:
        d = d * torch.rsqrt(d.square().sum(-1, keepdim=True) / s["H"] + EPS) * s["w_post"].double()
    if s["gate"] == "row":
        d = d * s["g"].double()[:, None]
    elif s["gate"] != "none":
        d = d * s["g"].double()
    r = s["r"].double() + float(np.float32(s["scale"])) * d
    if s["resid"] == "bf16":  # the next block reads the residual stream as it is kept
        kept = r.to(torch.bfloat16).double()
    else:
        kept = r
    x = kept * torch.rsqrt(kept.square().sum(-1, keepdim=True) / s["H"] + EPS) * s["w_pre"].double()
    return {"resid": r, "x_next": x}


def work(case):
    if case["op"] == "quant":  # the input, the packed rows and the values they stand for
        R, K = case["rows"], case["K"]
        return {"bytes": R * (K * SIZE[case["type"]] + row_bytes(K) + 2 * K), "flops": 4 * R * K}
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * row_bytes(K) + M * N * SIZE[case["out"]] + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    T, H = case["T"], case["H"]
    gate = {"none": 0, "channel": 4 * H, "row": 4 * T, "element": 2 * T * H}[case["gate"]]
    return {"bytes": T * H * (2 + 2 * SIZE[case["resid"]] + 2) + 4 * H * (2 if case["post"] else 1) + gate,
            "flops": 12 * T * H}
