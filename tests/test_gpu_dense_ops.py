"""The dense MXFP4 operators on the GPU against their definitions in 64 bits.

Quantised rows have to be equal bit for bit (one rounding of an exact quotient).  A product of small numbers whose
every partial sum 32 bits hold exactly has to be equal too, whatever its order; other products are off by at most
K * 2^-23 of the sum of the terms' magnitudes (each of the K additions of exact products rounds or truncates one
partial sum, which is no larger than that), the bias's addition and the rounding of y (bf16 2^-8, fp32 2^-24).
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from routed_expert_streaming_amd import _lib as L
from routed_expert_streaming_amd.runtime import (RMS_EPS, BlockNorms, MoEStack, MxLinear, pack_mx_expert,
                                                 quantise_mx)
from tests import mxkit

pytestmark = pytest.mark.gpu

HALF = {L.MOE_BF16: 2.0 ** -8, L.MOE_FP32: 2.0 ** -24}
DTYPE = {L.MOE_BF16: torch.bfloat16, L.MOE_FP16: torch.float16, L.MOE_FP32: torch.float32}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ quantisation
def special_blocks(dtype):
    """Blocks of 32 where the rule has an edge, in a type that holds them."""
    info = torch.finfo(dtype)
    tiny = info.smallest_normal
    step = tiny * info.eps  # the smallest subnormal
    ties = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.0, -0.0] + [0.0] * 20)
    blocks = [torch.zeros(32), -torch.zeros(32), ties, -ties, ties * 0.5, ties * 2.0 ** -10, ties * 2.0 ** 10,
              torch.full((32,), float(info.max)), torch.tensor([float(info.max)] + [1.0] * 31),
              torch.tensor([tiny] * 16 + [step] * 16), torch.tensor([step] + [0.0] * 31),
              torch.tensor([-3 * step, 5 * step, 7 * step] + [step] * 29), torch.tensor([tiny * 3] + [tiny / 2] * 31),
              torch.tensor([float("inf")] + [1.0] * 31), torch.tensor([1.0] * 31 + [float("nan")]),
              torch.tensor([-float("inf")] + [float("nan")] * 31), torch.full((32,), 6.0), torch.full((32,), 6.03125),
              torch.full((32,), 1.5), torch.tensor([1.501953125] + [1.0] * 31)]
    for e in range(-126, 128, 23):  # ties at scales all over the range
        if 2.0 ** e * 4 <= info.max and 2.0 ** e >= step:
            blocks.append(ties * 2.0 ** e)
    return torch.stack([b.to(dtype) for b in blocks])


@pytest.mark.parametrize("rule", ["floor", "fit"])
@pytest.mark.parametrize("kind", [L.MOE_BF16, L.MOE_FP16, L.MOE_FP32])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (5, 96), (7, 2080), (33, 512), (2, 6144), (257, 160)])
def test_quant(rows, K, kind, rule):
    g = torch.Generator().manual_seed(rows * 10007 + K)
    size = torch.exp(4 * torch.randn((rows, K // 32, 1), generator=g))  # blocks of very different sizes
    x = (torch.randn((rows, K // 32, 32), generator=g) * size).reshape(-1, 32).to(DTYPE[kind])
    sp = special_blocks(DTYPE[kind])
    n = min(len(sp), len(x))
    x[torch.randperm(len(x), generator=g)[:n]] = sp[:n]
    x = x.reshape(rows, K)
    check_quant(x, kind, rule)


def check_quant(x, kind, rule):
    rows, K = x.shape
    rb = mxkit.row_bytes(K)
    pad, gap = 16, 32  # bytes after a row of the input and of the output, which stay as they are
    wide = torch.zeros((rows, K + pad // x.element_size()), dtype=x.dtype, device="cuda")
    wide[:, :K] = x.cuda()
    out = torch.full((rows, rb + gap), 0xA5, dtype=torch.uint8, device="cuda")
    vals = torch.full((rows + 1, K), 7.0, dtype=torch.bfloat16, device="cuda")
    rule_id = L.MOE_MX_SCALE_FIT if rule == "fit" else L.MOE_MX_SCALE_FLOOR
    L.moe_mx_quant(wide, kind, K * x.element_size() + pad, rows, K, rule_id, out, rb + gap, vals,
                   torch.cuda.current_stream())
    codes, scales = mxkit.quantise(x.double().numpy(), rule)
    got = out.cpu().numpy()
    want = mxkit.pack(codes, scales)
    assert np.array_equal(got[:, K // 2:rb], want[:, K // 2:])  # scales and padding
    assert np.array_equal(got[:, :K // 2], want[:, :K // 2])
    assert (got[:, rb:] == 0xA5).all() and (vals[rows] == 7.0).all()
    ref = torch.from_numpy(mxkit.values(codes, scales)).to(torch.bfloat16)
    v = vals[:rows].cpu()
    assert torch.equal(v.isnan(), ref.isnan())
    assert torch.equal(v.view(torch.int16)[~ref.isnan()], ref.view(torch.int16)[~ref.isnan()])


@pytest.mark.parametrize("kind", [L.MOE_BF16, L.MOE_FP16, L.MOE_FP32])
def test_quant_edges(kind):
    for rule in ("floor", "fit"):
        check_quant(special_blocks(DTYPE[kind]), kind, rule)


def test_quant_every_bf16():
    """Each bf16 pattern once, each with one large neighbour in its block that puts it at some place of the grid."""
    bits = torch.arange(65536, dtype=torch.int32)
    v = bits.to(torch.int16).view(torch.bfloat16)
    x = torch.zeros((65536 // 31 + 1, 32), dtype=torch.bfloat16)
    flat = torch.zeros(x.shape[0] * 31, dtype=torch.bfloat16)
    flat[:65536] = v
    x[:, :31] = flat.reshape(-1, 31)
    x[:, 31] = x[:, :31].float().abs().nan_to_num(0, 0, 0).amax(1).to(torch.bfloat16)
    check_quant(x.reshape(-1, 32), L.MOE_BF16, "floor")


# ------------------------------------------------------------------ product
def run_matmul(a, kind, w, M, N, K, bias, y_type, w_gap=0, stream=None):
    """y [M, N] in float64; guard bytes around y's rows are checked."""
    size = 4 if y_type == L.MOE_FP32 else 2
    y = torch.full((M + 1, N + 3), 5.0, dtype=DTYPE[y_type], device="cuda")
    a_stride = mxkit.row_bytes(K) if kind == L.MOE_MXFP4 else 2 * K
    need = L.moe_mx_matmul_workspace_bytes(M, N, K, kind)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    L.moe_mx_matmul(a, kind, a_stride, w, mxkit.row_bytes(K) + w_gap, M, N, K, bias, y, y_type, size * (N + 3), ws,
                    need, stream if stream is not None else torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert (y[M] == 5.0).all() and (y[:, N:] == 5.0).all()
    assert (ws[need:] == 0xA5).all()
    return host(y[:M, :N])


def operand(rng, kind, R, K, low=126, high=128):
    """(device operand, its values): quarter-integers that bf16 holds, or MXFP4 rows with scales low .. high."""
    if kind == L.MOE_MXFP4:
        c, s = mxkit.random_rows(rng, R, K, low, high)
        return dev(mxkit.pack(c, s)), mxkit.values(c, s)
    v = rng.integers(-16, 17, (R, K)) * 0.25
    return dev(v, torch.bfloat16), v


def row_values(rows, K):
    """The values of MXFP4 rows on the device."""
    r = rows.cpu().numpy()
    codes = np.stack([r[:, :K // 2] & 15, r[:, :K // 2] >> 4], -1).reshape(r.shape[0], K).astype(np.int64)
    return mxkit.values(codes, r[:, K // 2:K // 2 + K // 32].astype(np.int64))


# M and N on both sides of every tile the kernels use, K with and without a short last group
M_SIZES = [1, 2, 3, 7, 15, 16, 17, 31, 33, 48, 64, 65, 100, 128, 129, 200, 257, 300]
N_SIZES = [1, 3, 16, 17, 31, 64, 65, 128, 130, 255, 257, 512, 700]
K_SIZES = [32, 64, 96, 128, 160, 256, 480, 512, 544, 1024, 1056]


@pytest.mark.parametrize("kind", [L.MOE_BF16, L.MOE_MXFP4])
@pytest.mark.parametrize("M", M_SIZES)
def test_matmul_exact_sums(M, kind):
    """Values are multiples of 1/4 (weights; activations alike) up to 12, so every product is a multiple of 1/16 up
    to 144 and every sum of at most 1056 of them is below 2^18: 22 bits, exact in any order."""
    rng = np.random.default_rng(M * 2 + kind)
    for i, N in enumerate(N_SIZES):
        K = K_SIZES[(i * 5 + M) % len(K_SIZES)]
        a, av = operand(rng, kind, M, K)
        wc, wsc = mxkit.random_rows(rng, N, K, 126, 128)
        gap = 16 * (i % 3)
        w = np.full((N, mxkit.row_bytes(K) + gap), 0xFF, np.uint8)  # NaN scales between the rows: never read
        w[:, :mxkit.row_bytes(K)] = mxkit.pack(wc, wsc)
        wv = mxkit.values(wc, wsc)
        b = rng.integers(-64, 65, N).astype(np.float32) if i % 2 else None
        want = av @ wv.T + (0.0 if b is None else b)
        got = run_matmul(a, kind, dev(w), M, N, K, None if b is None else dev(b), L.MOE_FP32, gap)
        assert np.array_equal(got, want), (M, N, K, kind, np.abs(got - want).max())
        got = run_matmul(a, kind, dev(w), M, N, K, None if b is None else dev(b), L.MOE_BF16, gap)
        ref = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16).double().numpy()
        assert np.array_equal(got, ref), (M, N, K, kind)


@pytest.mark.parametrize("kind", [L.MOE_BF16, L.MOE_MXFP4])
@pytest.mark.parametrize("M,N,K", [(2040, 6100, 1056), (2040, 4090, 1056), (1000, 2000, 544), (513, 1030, 1024),
                                   (130, 2100, 1056), (20, 5000, 1056), (64, 257, 1024), (3, 20011, 96),
                                   (8, 9001, 2048), (16, 4500, 544), (12, 5003, 96), (16, 9000, 1056), (1, 13000, 512),
                                   (16, 4200, 4608)])
def test_matmul_exact_sums_larger(M, N, K, kind):
    """As above, at sizes where the larger tiles, the parts of K and several tiles a workgroup are taken (4608
    terms of at most 144, or 48 where bf16 ones stop at 4: below 2^20 in 16ths, 24 bits)."""
    rng = np.random.default_rng(M + N)
    a, av = operand(rng, kind, M, K)
    c, s = mxkit.random_rows(rng, N, K, 126, 128)
    w, wv = dev(mxkit.pack(c, s)), mxkit.values(c, s)
    b = rng.integers(-64, 65, N).astype(np.float32)
    want = av @ wv.T + b
    assert np.array_equal(run_matmul(a, kind, w, M, N, K, dev(b), L.MOE_FP32), want)
    want = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16).double().numpy()
    assert np.array_equal(run_matmul(a, kind, w, M, N, K, dev(b), L.MOE_BF16), want)
    # rows of y that 16-byte stores cannot take, and ones that they can
    y = torch.full((M, (N + 7) // 8 * 8), 5.0, dtype=torch.bfloat16, device="cuda")
    need = L.moe_mx_matmul_workspace_bytes(M, N, K, kind)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    L.moe_mx_matmul(a, kind, a.stride(0) * a.element_size(), w, mxkit.row_bytes(K), M, N, K, dev(b), y, L.MOE_BF16,
                    2 * y.shape[1], ws, need, torch.cuda.current_stream())
    assert np.array_equal(host(y[:, :N]), want) and (y[:, N:] == 5.0).all()
    if need:
        with pytest.raises(L.MoEError) as ei:
            L.moe_mx_matmul(a, kind, a.stride(0) * a.element_size(), w, mxkit.row_bytes(K), M, N, K, None, y,
                            L.MOE_BF16, 2 * y.shape[1], ws, need - 1, torch.cuda.current_stream())
        assert ei.value.status == L.MOE_E_NOMEM


@pytest.mark.parametrize("kind", [L.MOE_BF16, L.MOE_MXFP4])
@pytest.mark.parametrize("M,far", [(3, "w"), (40, "w"), (150, "w"), (20, "a"), (70, "a"), (20, "both")])
def test_matmul_rows_far_apart(M, far, kind):
    """Operands whose rows lie 9 MB apart: views of larger buffers, beyond a tile's 32-bit offsets."""
    rng = np.random.default_rng(M)
    N, K, apart = 21, 544, 9 << 20
    a, av = operand(rng, kind, M, K)
    c, s = mxkit.random_rows(rng, N, K, 126, 128)
    w, wv = dev(mxkit.pack(c, s)), mxkit.values(c, s)

    def spread(t):
        rows = t.view(torch.uint8).reshape(t.shape[0], -1)
        wide = torch.zeros((t.shape[0], apart), dtype=torch.uint8, device="cuda")
        wide[:, :rows.shape[1]] = rows
        return wide
    a_far, w_far = far in ("a", "both"), far in ("w", "both")
    pa, pw = (spread(a) if a_far else a), (spread(w) if w_far else w)
    y = torch.zeros((M, N), device="cuda")
    need = L.moe_mx_matmul_workspace_bytes(M, N, K, kind)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    L.moe_mx_matmul(pa, kind, apart if a_far else a.stride(0) * a.element_size(), pw,
                    apart if w_far else mxkit.row_bytes(K), M, N, K, None, y, L.MOE_FP32, 4 * N, ws, need,
                    torch.cuda.current_stream())
    assert np.array_equal(host(y), av @ wv.T)


def check_product(got, av, wv, bias, K, y_type):
    want = av @ wv.T + (0.0 if bias is None else bias)
    terms = np.abs(av) @ np.abs(wv).T
    tol = K * 2.0 ** -23 * terms + (0 if bias is None else 2.0 ** -24 * (terms + np.abs(bias)))
    tol = tol + HALF[y_type] * (np.abs(want) + tol) + 1e-38
    worst = float((np.abs(got - want) / tol).max())
    assert worst <= 1.0, worst
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("y_type", [L.MOE_BF16, L.MOE_FP32])
@pytest.mark.parametrize("kind", [L.MOE_BF16, L.MOE_MXFP4])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (4, 1000, 6144), (16, 513, 2048), (32, 1536, 6144),
                                   (77, 300, 1568), (260, 520, 2080), (1024, 768, 1024), (2048, 2048, 512)])
def test_matmul_random(M, N, K, kind, y_type):
    rng = np.random.default_rng(M + N + K)
    if kind == L.MOE_MXFP4:
        c, s = mxkit.random_rows(rng, M, K, 118, 134)
        a, av = dev(mxkit.pack(c, s)), mxkit.values(c, s)
    else:
        a = dev(rng.standard_normal((M, K)), torch.bfloat16)
        av = host(a)
    c, s = mxkit.random_rows(rng, N, K, 116, 124)
    wv = mxkit.values(c, s)
    bias = rng.standard_normal(N).astype(np.float32) if M % 2 == 0 else None
    got = run_matmul(a, kind, dev(mxkit.pack(c, s)), M, N, K, None if bias is None else dev(bias), y_type)
    rel = check_product(got, av, wv, bias, K, y_type)
    print(f"M{M} N{N} K{K} kind {kind} y {y_type}: relative error {rel:.2e}")
    again = run_matmul(a, kind, dev(mxkit.pack(c, s)), M, N, K, None if bias is None else dev(bias), y_type)
    assert np.array_equal(got, again)  # fixed order: the same bits


@pytest.mark.parametrize("kind", [L.MOE_BF16, L.MOE_MXFP4])
@pytest.mark.parametrize("M", [1, 5, 40, 150, 300])
def test_matmul_special_values(M, kind):
    """Scale bytes 0, 1, 254 / 252 and 255; an activation row of infinities and NaN leaves the others alone."""
    rng = np.random.default_rng(M)
    N, K = 40, 288
    a, av = operand(rng, kind, M, K)
    wc, wsc = mxkit.random_rows(rng, N, K, 126, 128)
    wsc[3, 8] = 255            # a NaN block in the short last group: the whole output column
    wsc[7, :] = 252            # the largest that bf16 weights hold: one weight of 2^124
    wc[7, :], wc[7, 261] = 0, 1
    wsc[8, :] = 64
    wv = mxkit.values(wc, wsc)
    got = run_matmul(a, kind, dev(mxkit.pack(wc, wsc)), M, N, K, None, L.MOE_FP32)
    want = av @ wv.T
    assert np.isnan(got[:, 3]).all()
    plain = [n for n in range(N) if n != 3]
    assert np.array_equal(got[:, plain], want[:, plain])  # one power of two per column: the same exact sums, moved
    # the smallest scales, with activations 2^40 larger: sums in fp32's normal range, exact
    if kind == L.MOE_MXFP4:
        up = a.clone()
        up[:, K // 2:K // 2 + K // 32] += 40
    else:
        up = a * 2.0 ** 40
    low = wsc.copy()
    low[:] = rng.integers(0, 3, (N, 1))
    got_low = run_matmul(up, kind, dev(mxkit.pack(wc, low)), M, N, K, None, L.MOE_FP32)
    assert np.array_equal(got_low, (av * 2.0 ** 40) @ mxkit.values(wc, low).T)
    if M > 1:
        bad = a.clone()
        if kind == L.MOE_MXFP4:
            bad[0, K // 2:K // 2 + K // 32] = 255
        else:
            bad[0, ::2] = float("inf")
            bad[0, 1::2] = float("nan")
        hurt = run_matmul(bad, kind, dev(mxkit.pack(wc, wsc)), M, N, K, None, L.MOE_FP32)
        assert np.isnan(hurt[0]).all()
        assert np.array_equal(hurt[1:], got[1:], equal_nan=True)


# ------------------------------------------------------------------ norms around a block
def norm_case(rng, T, H, rt, post, gate, with_pre):
    add = dev(rng.standard_normal((T, H)) * 3, torch.bfloat16)
    resid = dev(rng.standard_normal((T, H)) * 5, DTYPE[rt])
    w_post = dev(1 + 0.3 * rng.standard_normal(H), torch.float32) if post == 2 else None
    w_pre = dev(1 + 0.3 * rng.standard_normal(H), torch.float32) if with_pre else None
    shape = {L.MOE_GATE_NONE: None, L.MOE_GATE_CHANNEL: (H,), L.MOE_GATE_ROW: (T,), L.MOE_GATE_ELEMENT: (T, H)}[gate]
    g = None if shape is None else dev(rng.standard_normal(shape),
                                       torch.bfloat16 if gate == L.MOE_GATE_ELEMENT else torch.float32)
    return add, resid, w_post, w_pre, g


def roundings(H):
    """Roundings of a sum of H squares here, at most: a thread's own (at least 256 threads), 6 of the wave, 15 of the
    waves, then mean, eps, root, reciprocal and three products."""
    return -(-H // 256) + 7 + 6 + 15 + 7


def check_norm(add, resid, out, x, post, w_post, g, gate, scale, w_pre, rt, eps):
    T, H = add.shape
    u = roundings(H) * 2.0 ** -24
    gh = None if g is None else (host(g)[:, None] if gate == L.MOE_GATE_ROW else host(g))
    wp = None if w_post is None else host(w_post)
    want = mxkit.block_norm(host(add), post > 0, wp, gh, float(np.float32(scale)), host(resid), eps)
    part = np.abs(want - host(resid))
    tol = u * part + 2.0 ** -24 * np.abs(want)
    if rt == L.MOE_BF16:
        tol = tol + 2.0 ** -8 * np.abs(want) + 2.0 ** -8 * tol
    worst = float((np.abs(host(out) - want) / (tol + 1e-38)).max())
    assert worst <= 1.0, worst
    if x is not None:
        nx = mxkit.norm(host(out), None if w_pre is None else host(w_pre), eps)  # of the stream as it is kept
        worst = float((np.abs(host(x) - nx) / ((2.0 ** -8 * (1 + u) + u) * np.abs(nx) + 1e-38)).max())
        assert worst <= 1.0, worst


@pytest.mark.parametrize("rt", [L.MOE_FP32, L.MOE_BF16])
@pytest.mark.parametrize("T,H", [(1, 4096), (3, 6144), (300, 1001), (2, 32), (5, 1), (1, 8200), (2, 40000), (257, 2048),
                                 (4, 16384), (1, 33333), (600, 8), (260, 5000)])
def test_block_norm(T, H, rt):
    rng = np.random.default_rng(T * 31 + H)
    eps, scale = 1e-6, 0.37
    for i, gate in enumerate((L.MOE_GATE_NONE, L.MOE_GATE_CHANNEL, L.MOE_GATE_ROW, L.MOE_GATE_ELEMENT)):
        for post in (0, 1, 2):  # none, without a weight, with one
            add, resid, w_post, w_pre, g = norm_case(rng, T, H, rt, post, gate, (i + post) % 2)
            out = torch.full((T + 1, H), 3.0, dtype=DTYPE[rt], device="cuda")
            x = torch.full((T + 1, H), 3.0, dtype=torch.bfloat16, device="cuda")
            s = torch.cuda.current_stream()
            before = resid.clone()
            L.moe_block_norm(add, post > 0, w_post, g, gate, scale, resid, out, rt, w_pre, T, H, eps, x, None, s)
            check_norm(add, resid, out[:T], x[:T], post, w_post, g, gate, scale, w_pre, rt, eps)
            assert torch.equal(resid, before) and (out[T] == 3.0).all() and (x[T] == 3.0).all()
            # in place, and without a next block
            L.moe_block_norm(add, post > 0, w_post, g, gate, scale, resid, resid, rt, w_pre, T, H, eps, None, None, s)
            assert torch.equal(resid, out[:T])
            # the pre-norm alone
            x2 = torch.empty_like(x[:T])
            L.moe_block_norm(None, 0, None, None, gate, scale, resid, None, rt, w_pre, T, H, eps, x2, None, s)
            assert torch.equal(x2, x[:T])


@pytest.mark.parametrize("T,H", [(1, 4096), (300, 2080), (5, 32), (2, 40000)])
@pytest.mark.parametrize("keep_x", [True, False])
def test_block_norm_writes_quantised_rows(T, H, keep_x):
    rng = np.random.default_rng(H)
    add, resid, w_post, w_pre, g = norm_case(rng, T, H, L.MOE_FP32, 2, L.MOE_GATE_CHANNEL, True)
    resid[0] = 0.0
    if T > 1:
        add[1] = 0.0
        resid[1, :] = float("nan")
    rb = mxkit.row_bytes(H)
    s = torch.cuda.current_stream()
    x, out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), torch.empty_like(resid)
    rows = torch.full((T + 1, rb), 0xA5, dtype=torch.uint8, device="cuda")
    L.moe_block_norm(add, 1, w_post, g, L.MOE_GATE_CHANNEL, 0.5, resid, out, L.MOE_FP32, w_pre, T, H, 1e-6, x, None, s)
    L.moe_block_norm(add, 1, w_post, g, L.MOE_GATE_CHANNEL, 0.5, resid, resid, L.MOE_FP32, w_pre, T, H, 1e-6,
                     torch.empty_like(x) if keep_x else None, rows, s)
    want = torch.empty((T, rb), dtype=torch.uint8, device="cuda")
    L.moe_mx_quant(x, L.MOE_BF16, 2 * H, T, H, L.MOE_MX_SCALE_FLOOR, want, rb, None, s)
    assert torch.equal(rows[:T], want) and (rows[T] == 0xA5).all()
    assert torch.equal(resid.view(torch.int32), out.view(torch.int32))


def test_block_norm_unaligned_and_degenerate_rows():
    rng = np.random.default_rng(3)
    T, H, eps = 7, 96, 1e-6
    add, resid, w_post, w_pre, g = norm_case(rng, T, H, L.MOE_FP32, 2, L.MOE_GATE_ELEMENT, True)
    add[2], resid[2] = 0.0, 0.0                       # a padded row: zeros stay zeros
    resid[3, 5] = float("inf")
    add[4, 1] = float("nan")
    s = torch.cuda.current_stream()
    out, x = torch.empty_like(resid), torch.empty_like(add)
    L.moe_block_norm(add, 1, w_post, g, L.MOE_GATE_ELEMENT, 1.0, resid, out, L.MOE_FP32, w_pre, T, H, eps, x, None, s)
    assert (out[2] == 0).all() and (x[2] == 0).all()
    assert out[3, 5].isinf() and x[3].isnan()[5] and (x[3, :5] == 0).all()  # inf / inf, finite / inf
    assert out[4].isnan().all() and x[4].isnan().all()
    ok = [0, 1, 5, 6]
    check_norm(add[ok], resid[ok], out[ok], x[ok], 2, w_post, g[ok], L.MOE_GATE_ELEMENT, 1.0, w_pre, L.MOE_FP32, eps)
    # the same values one element further on in memory
    def moved(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)
    out2, x2 = moved(out) * 0, moved(x) * 0
    out2, x2 = moved(out2), moved(x2)
    L.moe_block_norm(moved(add), 1, moved(w_post), moved(g), L.MOE_GATE_ELEMENT, 1.0, moved(resid), out2, L.MOE_FP32,
                     moved(w_pre), T, H, eps, x2, None, s)
    check_norm(add[ok], resid[ok], out2[ok], x2[ok], 2, w_post, g[ok], L.MOE_GATE_ELEMENT, 1.0, w_pre, L.MOE_FP32, eps)


def test_nothing_to_do():
    L.moe_mx_quant(None, L.MOE_BF16, 0, 0, 64, 0, None, 0, None, torch.cuda.current_stream())
    L.moe_mx_matmul(None, L.MOE_MXFP4, 0, None, 0, 0, 5, 64, None, None, L.MOE_BF16, 0)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ together
def dense_layer(add, resid, w_post, w_pre, w, N, K, rows, y, ws, stream):
    """norm -> quantised rows -> product, as a layer's dense half runs."""
    T = add.shape[0]
    L.moe_block_norm(add, 1, w_post, None, L.MOE_GATE_NONE, 0.5, resid, resid, L.MOE_FP32, w_pre, T, K, 1e-6, None, rows,
                     stream)
    L.moe_mx_matmul(rows, L.MOE_MXFP4, rows.shape[1], w, mxkit.row_bytes(K), T, N, K, None, y, L.MOE_BF16, 2 * N, ws,
                    ws.numel(), stream)


@pytest.mark.parametrize("T", [1, 6, 40, 300])
def test_layers_in_a_row_streams_and_graphs(T):
    """Two layers chained through the residual stream: against 64 bits step by step, on another stream, and captured
    into a graph that is replayed between eager runs."""
    rng = np.random.default_rng(T)
    K = N = 512
    s = torch.cuda.current_stream()
    w_post, w_pre = (dev(1 + 0.2 * rng.standard_normal(K), torch.float32) for _ in range(2))
    wf = [dev(rng.standard_normal((N, K)) * 0.05, torch.float32) for _ in range(2)]
    w = [torch.empty((N, mxkit.row_bytes(K)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for l in range(2):
        L.moe_mx_quant(wf[l], L.MOE_FP32, 4 * K, N, K, L.MOE_MX_SCALE_FIT, w[l], mxkit.row_bytes(K), None, s)
    add = dev(rng.standard_normal((T, K)), torch.bfloat16)
    resid0 = dev(rng.standard_normal((T, K)), torch.float32)

    def buffers():
        need = L.moe_mx_matmul_workspace_bytes(T, N, K, L.MOE_MXFP4)
        return dict(rows=torch.zeros((T, mxkit.row_bytes(K)), dtype=torch.uint8, device="cuda"),
                    y=torch.zeros((2, T, N), dtype=torch.bfloat16, device="cuda"), resid=resid0.clone(),
                    ws=torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda"))

    def step(b, stream):
        dense_layer(add, b["resid"], w_post, w_pre, w[0], N, K, b["rows"], b["y"][0], b["ws"], stream)
        dense_layer(b["y"][0], b["resid"], w_post, w_pre, w[1], N, K, b["rows"], b["y"][1], b["ws"], stream)

    one = buffers()
    step(one, s)
    torch.cuda.synchronize()
    # against 64 bits: the second layer from the stream as it was kept
    codes, scales = mxkit.quantise(host(wf[1]), "fit")
    wv = mxkit.values(codes, scales)
    assert np.array_equal(w[1].cpu().numpy(), mxkit.pack(codes, scales))
    check_product(host(one["y"][1]), row_values(one["rows"], K), wv, None, K, L.MOE_BF16)
    # another stream
    other = torch.cuda.Stream()
    two = buffers()
    other.wait_stream(s)
    step(two, other)
    other.synchronize()
    assert torch.equal(two["y"], one["y"]) and torch.equal(two["resid"], one["resid"])
    # a graph, replayed with eager work between
    three = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(three, torch.cuda.current_stream())
    for _ in range(4):
        three["resid"].copy_(resid0)
        three["y"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(three["y"], one["y"]) and torch.equal(three["resid"], one["resid"])
        two["resid"].copy_(resid0)
        step(two, s)
        torch.cuda.synchronize()
        assert torch.equal(two["y"], one["y"])


def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(11)
    K = 4096
    streams = [torch.cuda.Stream() for _ in range(4)]
    data = []
    for M, N in ((3, 1000), (60, 1000), (128, 2048), (256, 4096)):
        c, sc = mxkit.random_rows(rng, N, K, 120, 124)
        a = dev(rng.standard_normal((M, K)), torch.bfloat16)
        need = L.moe_mx_matmul_workspace_bytes(M, N, K, L.MOE_BF16)
        data.append((M, N, a, dev(mxkit.pack(c, sc)), torch.zeros((M, N), device="cuda"),
                     torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda"), need))
    assert any(d[-1] for d in data)  # K in parts somewhere

    def go(d, stream):
        M, N, a, w, y, ws, need = d
        L.moe_mx_matmul(a, L.MOE_BF16, 2 * K, w, mxkit.row_bytes(K), M, N, K, None, y, L.MOE_FP32, 4 * N, ws, need, stream)

    want = []
    for d in data:
        go(d, torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append(d[4].clone())
        check_product(host(d[4]), host(d[2]), row_values(d[3], K), None, K, L.MOE_FP32)
        d[4].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for d, st in zip(data, streams):
            go(d, st)
    torch.cuda.synchronize()
    for d, v in zip(data, want):
        assert torch.equal(d[4], v)
    # each in a graph of its own, all replayed together between eager calls
    graphs = []
    for d in data:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            go(d, torch.cuda.current_stream())
    for _ in range(3):
        for d in data:
            d[4].zero_()
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for d, v in zip(data, want):
            assert torch.equal(d[4], v)
            go(d, torch.cuda.current_stream())


def test_quantised_experts_in_the_routed_ffn():
    """A bf16 checkpoint's expert packed into a slab by the row quantiser (gate and up rows interleaved) runs through
    the routed FFN, and its gate matrix through the dense product, where it lies."""
    rng = np.random.default_rng(7)
    H, I, E, T, k = 256, 128, 4, 5, 2
    s = torch.cuda.current_stream()
    rb, rbi = mxkit.row_bytes(H), mxkit.row_bytes(I)
    pool = torch.zeros((E, L.moe_expert_bytes_mx(H, I)), dtype=torch.uint8, device="cuda")
    gate = None
    for e in range(E):
        mats = [dev(rng.standard_normal(shape) * 0.05, torch.bfloat16) for shape in ((I, H), (I, H), (H, I))]
        L.moe_mx_quant(mats[0], L.MOE_BF16, 2 * H, I, H, L.MOE_MX_SCALE_FLOOR, pool[e], 2 * rb, None, s)
        L.moe_mx_quant(mats[1], L.MOE_BF16, 2 * H, I, H, L.MOE_MX_SCALE_FLOOR, pool[e][rb:], 2 * rb, None, s)
        L.moe_mx_quant(mats[2], L.MOE_BF16, 2 * I, H, I, L.MOE_MX_SCALE_FLOOR, pool[e][2 * I * rb:], rbi, None, s)
        if e == 1:
            gate = mats[0]
    x = dev(rng.standard_normal((T, H)), torch.bfloat16)
    idx = dev(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32))
    table = dev(np.array([pool[e].data_ptr() for e in range(E)], np.int64))
    y = torch.zeros((T * k, H), device="cuda")
    nb = L.moe_expert_ffn_workspace_bytes(T, H, I, E, k, False)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    L.moe_expert_ffn_fmt(x, T, H, I, E, idx, k, table, None, None, y, ws, nb, L.MOE_FFN_AUTO, 1, s)
    torch.cuda.synchronize()
    slabs = [pool[e].cpu().numpy() for e in range(E)]
    got = host(y).reshape(T, k, H)
    for t in range(T):
        for j in range(k):
            ref = oracle.expert_ffn(slabs[int(idx[t, j])], H, I, host(x)[t], 1)[3]
            assert np.abs(got[t, j] - ref).max() <= 2e-2 * np.abs(ref).max()
    # the gate matrix inside the slab as the dense product's weights
    d = torch.zeros((T, I), device="cuda")
    L.moe_mx_matmul(x, L.MOE_BF16, 2 * H, pool[1], 2 * rb, T, I, H, None, d, L.MOE_FP32, 4 * I, None, 0, s)
    torch.cuda.synchronize()
    wv = mxkit.values(*mxkit.quantise(host(gate), "floor"))
    check_product(host(d), host(x), wv, None, H, L.MOE_FP32)


# ------------------------------------------------------------------ through the runtime
def test_quantise_mx_refuses_a_small_or_foreign_out():
    w = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    for out, stride in ((torch.zeros(2 * 48 + 47, dtype=torch.uint8, device="cuda"), 48),
                        (torch.zeros(3 * 48, dtype=torch.uint8), 48),
                        (torch.zeros(3 * 48, dtype=torch.int8, device="cuda"), 48),
                        (torch.zeros((3, 96), dtype=torch.uint8, device="cuda")[:, :48], 96)):
        with pytest.raises(ValueError):
            quantise_mx(w, out, stride)
    with pytest.raises(L.MoEError):
        quantise_mx(w, torch.zeros(3 * 48, dtype=torch.uint8, device="cuda"), 32)  # rows would overlap
    out = torch.zeros(2 * 64 + 48, dtype=torch.uint8, device="cuda")
    quantise_mx(w, out, 64)
    assert torch.equal(out[64:64 + 48], quantise_mx(w)[1])


def test_pack_mx_expert():
    rng = np.random.default_rng(9)
    H, I = 96, 64
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        mats = [dev(rng.standard_normal(s) * 0.1, dtype) for s in ((I, H), (I, H), (H, I))]
        pool = torch.full((3, L.moe_expert_bytes_mx(H, I)), 0xA5, dtype=torch.uint8, device="cuda")
        assert pack_mx_expert(*mats, slab=pool[1]).data_ptr() == pool[1].data_ptr()
        fresh = pack_mx_expert(*mats)
        assert torch.equal(fresh, pool[1]) and (pool[0] == 0xA5).all() and (pool[2] == 0xA5).all()
        for which, m in enumerate(mats):
            want = mxkit.values(*mxkit.quantise(host(m), "floor"))
            assert np.array_equal(oracle.dequant(fresh.cpu().numpy(), H, I, which, 1), want)


@pytest.mark.parametrize("quantise_input", [False, True])
def test_mx_linear(quantise_input):
    rng = np.random.default_rng(4)
    N, K = 330, 544
    weight = dev(rng.standard_normal((N, K)) * 0.05, torch.bfloat16)
    bias = dev(rng.standard_normal(N), torch.bfloat16)
    wide = torch.zeros((N, K + 32), dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = weight
    for out_dtype, y_type in ((torch.bfloat16, L.MOE_BF16), (torch.float32, L.MOE_FP32)):
        lin = MxLinear(wide[:, :K], bias, quantise_input, out_dtype)  # a view with rows further apart
        assert torch.equal(lin.rows, quantise_mx(weight))
        wv = mxkit.values(*mxkit.quantise(host(weight), "floor"))
        for shape in ((1, K), (3, 5, K), (70, K), (0, K)):
            x = dev(rng.standard_normal(shape), torch.bfloat16)
            y = lin(x)
            assert y.shape == (*shape[:-1], N) and y.dtype == out_dtype
            if shape[0] == 0:
                continue
            xv = host(x).reshape(-1, K)
            if quantise_input:
                xv = mxkit.values(*mxkit.quantise(xv, "floor"))
                assert torch.equal(lin(quantise_mx(x.reshape(-1, K))).reshape(y.shape), y)
            check_product(host(y).reshape(-1, N), xv, wv, host(bias), K, y_type)
        every = dev(rng.standard_normal((6, K)), torch.bfloat16)
        assert torch.equal(lin(every[::2]), lin(every[::2].contiguous()))  # rows apart
        for bad in (every.float(), every[:, :32], every.cpu()):
            with pytest.raises(ValueError):
                lin(bad)


@pytest.mark.parametrize("post,gate", [(True, True), (False, True), (True, False), (False, False)])
def test_chained_layers_with_norms(post, gate):
    """A chained step with learned norms: every layer's input against the formula in 64 bits on the layers' own
    outputs; the same step without norms is left as it was."""
    st = MoEStack(synth.get("tiny", layers=3))
    try:
        rng = np.random.default_rng(1)
        Lyr, T, H = st.L, st.T, st.H
        norms = BlockNorms(dev(1 + 0.2 * rng.standard_normal((Lyr, H)), torch.float32),
                           dev(1 + 0.2 * rng.standard_normal((Lyr, H)), torch.float32) if post else None,
                           dev(rng.random((Lyr, H)), torch.float32) if gate else None, 0.5)
        resid, xs = st.chain_buffers()
        out, h0 = st.new_output(), st.make_inputs(0)[0]
        st.forward_chained(h0, xs, resid, out, norms=norms)
        torch.cuda.synchronize()
        r = host(h0)
        u = roundings(H) * 2.0 ** -24
        err = np.zeros_like(r)  # how far the stream may be from these 64-bit values
        for l in range(Lyr):
            want = mxkit.norm(r, host(norms.pre[l]), RMS_EPS)
            # an error of the stream moves x by as much as it is of the row's root mean square
            rms = np.sqrt((r * r).mean(1, keepdims=True))
            moved = (err + np.abs(r) * err.max(1, keepdims=True) / rms) / rms * np.abs(host(norms.pre[l]))
            tol = (2.0 ** -8 * (1 + u) + u) * np.abs(want) + 2 * moved
            assert (np.abs(host(xs[l]) - want) <= tol).all(), l
            if l + 1 < Lyr:
                d = host(out[l])
                nxt = mxkit.block_norm(d, post, host(norms.post[l]) if post else None,
                                       host(norms.gate[l]) if gate else None, 0.5, r, RMS_EPS)
                err = err + u * np.abs(nxt - r) + 2.0 ** -24 * (np.abs(nxt) + err)
                r = nxt
        assert (np.abs(host(resid) - r) <= err).all()
        # against the plain chain: unit weights, no gate, scale 1 give the same layers up to the sums' order
        resid1, xs1 = st.chain_buffers()
        out1 = st.new_output()
        st.forward_chained(h0, xs1, resid1, out1)
        ones = BlockNorms(torch.ones((Lyr, H), device="cuda"))
        resid2, xs2 = st.chain_buffers()
        st.forward_chained(h0, xs2, resid2, out, norms=ones)
        torch.cuda.synchronize()
        assert (np.abs(host(xs2[0]) - host(xs1[0])) <= 2.0 ** -7 * np.abs(host(xs1[0]))).all()  # one bf16 step
        for bad in (BlockNorms(norms.pre[:1]), BlockNorms(norms.pre.double()), BlockNorms(norms.pre, norms.pre.t())):
            with pytest.raises(ValueError):
                st.forward_chained(h0, xs2, resid2, out, norms=bad)
    finally:
        st.close()


# ------------------------------------------------------------------ offsets past 32 bits
def test_offsets_past_32_bits():
    """Operands beyond 4 GiB: their last rows give what a small call on those rows gives."""
    s = torch.cuda.current_stream()
    g = torch.Generator(device="cuda").manual_seed(2)
    K = 8192
    rb = mxkit.row_bytes(K)
    # weights: 1,100,000 rows of 4352 bytes
    N, tail = 1100000, 70
    w = torch.randint(0, 256, (N, rb), dtype=torch.uint8, device="cuda", generator=g)
    w[:, K // 2:] = 120
    wv = row_values(w[-tail:], K)
    for M, kind in ((2, L.MOE_BF16), (2, L.MOE_MXFP4), (40, L.MOE_MXFP4), (130, L.MOE_BF16)):
        rng = np.random.default_rng(M)
        a, av = operand(rng, kind, M, K)
        y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
        need = L.moe_mx_matmul_workspace_bytes(M, N, K, kind)
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        L.moe_mx_matmul(a, kind, a.stride(0) * a.element_size(), w, rb, M, N, K, None, y, L.MOE_BF16, 2 * N, ws, need, s)
        check_product(host(y[:, -tail:]), av, wv, None, K, L.MOE_BF16)
    del w, y, ws
    # activations and output: 300,000 rows
    M, N = 300000, 8200
    a = torch.randint(0, 256, (M, rb), dtype=torch.uint8, device="cuda", generator=g)
    a[:, K // 2:] = 124
    c, sc = mxkit.random_rows(np.random.default_rng(1), N, K, 118, 121)
    w = dev(mxkit.pack(c, sc))
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    assert L.moe_mx_matmul_workspace_bytes(M, N, K, L.MOE_MXFP4) == 0
    L.moe_mx_matmul(a, L.MOE_MXFP4, rb, w, rb, M, N, K, None, y, L.MOE_BF16, 2 * N, None, 0, s)
    check_product(host(y[-5:]), row_values(a[-5:], K), mxkit.values(c, sc), None, K, L.MOE_BF16)
    del a, y, w
    # quantiser and norm: 300,000 x 8192
    x = torch.randn((M, K), dtype=torch.bfloat16, device="cuda", generator=g)
    rows = torch.empty((M, rb), dtype=torch.uint8, device="cuda")
    vals = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    L.moe_mx_quant(x, L.MOE_BF16, 2 * K, M, K, L.MOE_MX_SCALE_FLOOR, rows, rb, vals, s)
    codes, scales = mxkit.quantise(host(x[-2:]), "floor")
    assert np.array_equal(rows[-2:].cpu().numpy(), mxkit.pack(codes, scales))
    assert np.array_equal(host(vals[-2:]), mxkit.values(codes, scales))
    resid = torch.randn((M, K), device="cuda", generator=g)
    out = torch.empty_like(resid)
    L.moe_block_norm(x, 1, None, None, L.MOE_GATE_NONE, 0.5, resid, out, L.MOE_FP32, None, M, K, 1e-6, vals, rows, s)
    check_norm(x[-3:], resid[-3:], out[-3:], vals[-3:], 1, None, None, L.MOE_GATE_NONE, 0.5, None, L.MOE_FP32, 1e-6)
    codes, scales = mxkit.quantise(host(vals[-1:]), "floor")
    assert np.array_equal(rows[-1:].cpu().numpy(), mxkit.pack(codes, scales))
