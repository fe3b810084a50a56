"""The FP8 operators on the GPU against their definitions in 64 bits.

Codes and scales have to be equal bit for bit.  A product whose every partial sum 32 bits hold exactly has to be equal
too; other products are off by at most fp8kit.sum_error(K) of the sum of the terms' magnitudes, with y in bf16 by what
the FP8 matrix cores cut (fp8kit.cores_error), the bias's addition (2^-24 of the sum) and the rounding of y (bf16 2^-8,
fp32 2^-24).
"""
import numpy as np
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from tests import fp8kit

pytestmark = pytest.mark.gpu

HALF = {L.MOE_BF16: 2.0 ** -8, L.MOE_FP32: 2.0 ** -24}
DTYPE = {L.MOE_BF16: torch.bfloat16, L.MOE_FP16: torch.float16, L.MOE_FP32: torch.float32}
RULE = {"amax": L.MOE_FP8_SCALE_AMAX, "pow2": L.MOE_FP8_SCALE_POW2}


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


# ------------------------------------------------------------------ quantisation
def check_quant(x, kind, block_rows, rule):
    """x [rows, K] of a torch type; bytes around the outputs' rows have to stay."""
    rows, K = x.shape
    wide = torch.full((rows, K + 16), 3.0, dtype=x.dtype, device="cuda")
    wide[:, :K] = x.cuda()
    R, C = -(-rows // block_rows), fp8kit.blocks(K)
    codes = torch.full((rows + 1, K + 32), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((R + 1, C + 3), 7.0, device="cuda")
    L.moe_fp8_quant(wide, kind, (K + 16) * x.element_size(), rows, K, block_rows, RULE[rule], codes, K + 32, scales,
                    4 * (C + 3), torch.cuda.current_stream())
    rc, rs = fp8kit.quantise(x.double().numpy(), block_rows, rule)
    got_c, got_s = codes.cpu().numpy(), scales.cpu().numpy()
    assert (got_c[:, K:] == 0xA5).all() and (got_c[rows] == 0xA5).all()
    assert (got_s[:, C:] == 7.0).all() and (got_s[R] == 7.0).all()
    assert np.array_equal(got_s[:R, :C], rs, equal_nan=True)
    assert np.array_equal(got_c[:rows, :K], rc)


@pytest.mark.parametrize("rule", ["amax", "pow2"])
@pytest.mark.parametrize("kind", [L.MOE_BF16, L.MOE_FP16, L.MOE_FP32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 128), (5, 144), (1, 4096), (7, 2080), (129, 272), (257, 112)])
def test_quant(rows, K, block_rows, kind, rule):
    g = torch.Generator().manual_seed(rows * 10007 + K)
    size = torch.exp(3 * torch.randn((rows, (K + 15) // 16, 1), generator=g))
    x = (torch.randn((rows, (K + 15) // 16, 16), generator=g) * size).reshape(rows, -1)[:, :K].to(DTYPE[kind])
    check_quant(x, kind, block_rows, rule)


@pytest.mark.parametrize("rule", ["amax", "pow2"])
@pytest.mark.parametrize("kind", [L.MOE_BF16, L.MOE_FP16, L.MOE_FP32])
def test_quant_edges(kind, rule):
    """Zeros, infinities, NaN, the type's extremes and subnormals, ties at every size, largest magnitudes around 448's
    powers of two."""
    info = torch.finfo(DTYPE[kind])
    step = info.smallest_normal * info.eps
    grid = torch.from_numpy(fp8kit.GRID)
    ties = (grid[1:] + grid[:-1]) / 2
    rows = [torch.zeros(128), -torch.zeros(128), torch.full((128,), info.max), torch.full((128,), step),
            torch.cat([torch.tensor([info.max]), torch.full((127,), step)]),
            torch.cat([torch.tensor([float("inf")]), torch.ones(127)]),
            torch.cat([torch.ones(127), torch.tensor([float("nan")])]),
            torch.cat([torch.ones(100), torch.full((28,), -float("inf"))]),
            torch.arange(128) * step, torch.arange(128) * -37 * step, grid.repeat(2)[:128], -grid.repeat(2)[:128],
            torch.cat([torch.tensor([448.0]), ties[:126], torch.zeros(1)]),
            torch.cat([torch.tensor([-448.0]), -ties[:126], torch.zeros(1)])]
    for e in range(-140, 125, 11):
        if step <= 2.0 ** e and 450 * 2.0 ** e <= info.max:
            rows += [torch.cat([torch.tensor([448.0]), ties[:126], torch.zeros(1)]) * 2.0 ** e,
                     torch.cat([torch.tensor([449.0]), ties[:126], torch.zeros(1)]).double() * 2.0 ** e,
                     torch.full((128,), 2.0 ** e)]
    x = torch.stack([r.double() for r in rows]).to(DTYPE[kind])
    check_quant(x, kind, 1, rule)
    for r in x:  # each as a block of rows of its own
        check_quant(torch.stack([r, torch.zeros_like(r)]), kind, 128, rule)


def test_quant_rounds_the_true_quotient():
    """Values a few ulps to either side of every border between two codes, at scales that are no powers of two."""
    rng = np.random.default_rng(3)
    grid = fp8kit.GRID
    ties = (grid[1:] + grid[:-1]) / 2
    rows = []
    for top in np.concatenate([rng.uniform(1, 2, 40) * 2.0 ** rng.integers(-120, 100, 40), [2.0 ** -130, 2.0 ** -118]]):
        top = np.float32(top)
        s = np.float64(max(np.float32(np.float64(top) / 448), np.float32(2.0 ** -126)))
        v = (ties * s).astype(np.float32)
        for d in range(-2, 3):
            near = v.copy()
            for _ in range(abs(d)):
                near = np.nextafter(near, np.float32(np.inf if d > 0 else 0))
            rows.append(np.concatenate([[top], near, [0]]).astype(np.float32))
    x = torch.from_numpy(np.stack(rows))
    check_quant(x, L.MOE_FP32, 1, "amax")


def test_quant_many_rows():
    """More than one launch takes, and rows beyond 4 GiB of input."""
    rows, K = (1 << 26) + 3, 16  # 2^26 rows of 16 lanes are one launch
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    x[-1] = 2.0
    x[(1 << 26) - 1] = 4.0
    codes = torch.empty((rows, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, 1), device="cuda")
    L.moe_fp8_quant(x, L.MOE_BF16, 2 * K, rows, K, 1, L.MOE_FP8_SCALE_POW2, codes, K, scales, 4,
                    torch.cuda.current_stream())
    top = codes.amax(1)
    assert top[-1] == 0x78 and top[(1 << 26) - 1] == 0x78  # 256 = 2 / 2^-7 = 4 / 2^-6: exponent field 15, mantissa 0
    assert scales[-1, 0] == 2.0 ** -7 and scales[(1 << 26) - 1, 0] == 2.0 ** -6
    top[-1] = top[(1 << 26) - 1] = 0
    assert not top.any() and (scales == 1).sum() == rows - 2


# ------------------------------------------------------------------ product
def small_operand(rng, R, K, block_rows):
    """Codes of whole numbers -8 .. 8 and scales 2^-1 .. 2^1: sums of up to 2^15 such products are exact in 32 bits."""
    v = rng.integers(-8, 9, (R, K)).astype(np.float64)
    codes = (fp8kit.nearest(np.abs(v)) + 128 * (v < 0)).astype(np.uint8)
    scales = 2.0 ** rng.integers(-1, 2, (-(-R // block_rows), fp8kit.blocks(K)))
    return codes, scales.astype(np.float32)


def random_operand(rng, R, K, block_rows):
    codes = rng.integers(0, 256, (R, K)).astype(np.uint8)
    codes[codes & 127 == 127] = 5
    return codes, np.exp(2 * rng.standard_normal((-(-R // block_rows), fp8kit.blocks(K)))).astype(np.float32)


def run_matmul(a, sa, w, sw, M, N, K, bias, y_type, a_gap=0, w_gap=0, stream=None):
    """y [M, N] in float64 from host operands, with gaps between the rows of both, and bytes around y's rows checked."""
    def wide(c, gap):
        buf = np.full((c.shape[0], c.shape[1] + gap), 0x7F, np.uint8)  # NaN behind the rows
        buf[:, :c.shape[1]] = c
        return dev(buf)
    y = torch.full((M + 1, N + 3), 5.0, dtype=DTYPE[y_type], device="cuda")
    size = y.element_size()
    need = L.moe_fp8_matmul_workspace_bytes(M, N, K, L.MOE_FP8)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    pa, pw = fp8kit.padded(sa), np.concatenate([sw, np.full((sw.shape[0], 1), np.nan, np.float32)], axis=1)
    L.moe_fp8_matmul(wide(a, a_gap), L.MOE_FP8, K + a_gap, dev(pa), 4 * pa.shape[1], wide(w, w_gap), K + w_gap, dev(pw),
                     4 * pw.shape[1], M, N, K, None if bias is None else dev(bias, torch.float32), y, y_type,
                     size * (N + 3), ws, need, torch.cuda.current_stream() if stream is None else stream)
    torch.cuda.synchronize()
    assert (y[M] == 5.0).all() and (y[:, N:] == 5.0).all() and (ws[need:] == 0xA5).all()
    return y[:M, :N].double().cpu().numpy()


SHAPES = [(1, 1, 16), (1, 16, 128), (1, 130, 4096), (2, 128, 144), (5, 33, 1040), (15, 257, 256), (16, 64, 2080),
          (17, 129, 400), (31, 48, 1552), (32, 300, 640), (33, 256, 128), (48, 100, 1024), (64, 384, 528), (65, 130, 272),
          (100, 1001, 1568), (129, 128, 2048), (200, 640, 112), (256, 256, 384), (257, 257, 1104), (300, 513, 3200),
          (513, 129, 96), (1000, 72, 560), (40, 2100, 800)]


@pytest.mark.parametrize("y_type", [L.MOE_BF16, L.MOE_FP32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_exact(M, N, K, y_type):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    a, sa = small_operand(rng, M, K, 1)
    w, sw = small_operand(rng, N, K, 128)
    bias = rng.integers(-50, 51, N).astype(np.float64) if N % 2 else None
    got = run_matmul(a, sa, w, sw, M, N, K, bias, y_type, 16 * (M % 3), 16 * (N % 3))
    want = fp8kit.values(a, sa, 1) @ fp8kit.values(w, sw, 128).T
    if bias is not None:
        want = want + bias
    want = torch.from_numpy(want).to(DTYPE[y_type]).double().numpy()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(M, N, K):
    rng = np.random.default_rng(M + N * 13 + K * 17)
    a, sa = random_operand(rng, M, K, 1)
    w, sw = random_operand(rng, N, K, 128)
    bias = rng.standard_normal(N) if M % 2 else None
    va, vw = fp8kit.values(a, sa, 1), fp8kit.values(w, sw, 128)
    want, mag = va @ vw.T, np.abs(va) @ np.abs(vw).T
    if bias is not None:
        bias = bias.astype(np.float32).astype(np.float64)
        want, mag = want + bias, mag + np.abs(bias)
    for y_type in (L.MOE_BF16, L.MOE_FP32):
        got = run_matmul(a, sa, w, sw, M, N, K, bias, y_type)
        err = (fp8kit.sum_error(K) + fp8kit.cores_error(y_type == L.MOE_BF16) + 2.0 ** -24) * mag
        assert (np.abs(got - want) <= err + HALF[y_type] * (np.abs(want) + err)).all()


@pytest.mark.parametrize("M,N,K", [(1, 48, 256), (20, 144, 1040), (150, 300, 400), (600, 520, 1040)])
def test_matmul_nan(M, N, K):
    """NaN codes and scales reach the outputs they enter and no others; the largest values stay finite."""
    rng = np.random.default_rng(1)
    a, sa = small_operand(rng, M, K, 1)
    w, sw = small_operand(rng, N, K, 128)
    a[M - 1, K - 1] = 0x7F
    w[N // 2, 0] = 0xFF
    sa[0, fp8kit.blocks(K) - 1] = np.nan
    sw[fp8kit.blocks(N) - 1, 0] = np.nan
    got = run_matmul(a, sa, w, sw, M, N, K, None, L.MOE_FP32)
    want = fp8kit.values(a, sa, 1) @ fp8kit.values(w, sw, 128).T
    assert np.array_equal(got, want, equal_nan=True)
    a[:], w[:], sa[:], sw[:] = 0x7E, 0xFE, 2.0, 0.5
    got = run_matmul(a, sa, w, sw, M, N, K, None, L.MOE_FP32)
    assert np.abs(got / (-448.0 ** 2 * K) - 1).max() <= fp8kit.sum_error(K) + 2.0 ** -24


@pytest.mark.parametrize("M,N,K", [(1, 130, 4096), (4, 300, 1040), (16, 64, 272), (17, 129, 528), (64, 256, 400),
                                   (130, 520, 640), (700, 300, 272)])
def test_matmul_quantises_bf16(M, N, K):
    """bf16 activations give the bits that their codes from moe_fp8_quant give; rows with gaps, an infinite row."""
    rng = np.random.default_rng(M + K)
    w, sw = random_operand(rng, N, K, 128)
    x = torch.randn((M, K + 8), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16)
    x[:, :8] *= 30
    if M > 3:
        x[2, 3] = float("inf")
        x[3, :K] = 0
    xd = x.cuda()
    codes = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    srow = (fp8kit.blocks(K) + 3) // 4 * 4
    scales = torch.empty((M, srow), device="cuda")
    s = torch.cuda.current_stream()
    L.moe_fp8_quant(xd, L.MOE_BF16, 2 * (K + 8), M, K, 1, L.MOE_FP8_SCALE_AMAX, codes, K, scales, 4 * srow, s)
    wd, swd = dev(w), dev(sw)
    out = []
    for a, kind, stride, sc in ((xd, L.MOE_BF16, 2 * (K + 8), None), (codes, L.MOE_FP8, K, scales)):
        y = torch.empty((M, N), device="cuda")
        need = L.moe_fp8_matmul_workspace_bytes(M, N, K, kind)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        L.moe_fp8_matmul(a, kind, stride, sc, 4 * srow, wd, K, swd, 4 * fp8kit.blocks(K), M, N, K, None, y, L.MOE_FP32,
                         4 * N, ws, need, s)
        out.append(y.cpu().numpy())
    # beyond 16 rows the same kernel multiplies the same codes; up to there one that quantises them itself adds the blocks'
    # sums in another order (one chain of fused additions, or parts that are joined): each is within sum_error
    if M > 16:
        assert np.array_equal(out[0], out[1], equal_nan=True)
    rc, rs = fp8kit.quantise(x[:, :K].double().numpy())
    va, vw = fp8kit.values(rc, rs, 1), fp8kit.values(w, sw, 128)
    want, mag = va @ vw.T, np.abs(va) @ np.abs(vw).T
    ok = ~np.isnan(want)
    for y in out:
        assert np.array_equal(ok, ~np.isnan(y))
        assert (np.abs(y - want) <= (fp8kit.sum_error(K) + 2.0 ** -24) * mag + 2.0 ** -24 * np.abs(want))[ok].all()


def test_matmul_streams_and_graphs():
    rng = np.random.default_rng(77)
    for M, N, K in ((1, 512, 1024), (24, 384, 640), (300, 520, 400)):
        w, sw = random_operand(rng, N, K, 128)
        wd, swd = dev(w), dev(sw)
        x = [torch.randn((M, K), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in range(2)]
        y = [torch.zeros((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        need = L.moe_fp8_matmul_workspace_bytes(M, N, K, L.MOE_BF16)
        ws = [torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") for _ in range(2)]

        def call(i, stream=None):
            L.moe_fp8_matmul(x[i], L.MOE_BF16, 2 * K, None, 0, wd, K, swd, 4 * fp8kit.blocks(K), M, N, K, None, y[i],
                             L.MOE_BF16, 2 * N, ws[i], need, torch.cuda.current_stream() if stream is None else stream)
        want = []
        for i in range(2):
            call(i)
            torch.cuda.synchronize()
            want.append(y[i].clone())
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(4):
            for i in range(2):
                y[i].zero_()
            torch.cuda.synchronize()
            for i in range(2):
                call(i, streams[i])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(y, want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(0)
            call(1)
        for _ in range(3):
            for i in range(2):
                y[i].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(y, want))
            call(0)
            torch.cuda.synchronize()


# ------------------------------------------------------------------ experts
class Experts:
    """E experts (and a shared one) of random codes, on the host and as slabs on the device."""

    def __init__(self, seed, H, I, E, shared):
        rng = np.random.default_rng(seed)
        self.H, self.I, self.E = H, I, E
        self.parts = []
        for _ in range(E + shared):
            mats = []
            for R, K in ((I, H), (I, H), (H, I)):
                w = (rng.standard_normal((R, K)) * (1.5 / K ** 0.5)).astype(np.float32).astype(np.float64)
                mats.append(fp8kit.quantise(w, 128, "amax"))
            self.parts.append(mats)
        n = L.moe_expert_bytes_fp8(H, I)
        slabs = [fp8kit.slab(p) for p in self.parts]
        assert all(len(s) == n for s in slabs)
        self.slabs = dev(np.stack(slabs))
        order = rng.permutation(E)  # the experts lie in the pool in any order
        pool = torch.empty((E, n), dtype=torch.uint8, device="cuda")
        pool[torch.from_numpy(order).cuda()] = self.slabs[:E]
        self.pool = pool
        self.table = dev(pool.data_ptr() + n * order.astype(np.int64))
        self.shared = self.slabs[E] if shared else None


def routing(rng, T, E, k, busy=0):
    """Each token's k experts; the first `busy` tokens all take expert 0 first."""
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    for t in range(min(busy, T)):
        at = np.nonzero(idx[t] == 0)[0]
        if len(at):
            idx[t, at[0]] = idx[t, 0]
        idx[t, 0] = 0
    return idx.astype(np.int32)


def reference(ex, x, idx, mask=None):
    """(y, error bound) rows of pairs and of the shared expert, NaN for pairs that are masked off."""
    T, k = idx.shape
    q, s = fp8kit.quantise(x)
    xq = fp8kit.values(q, s, 1)
    rows = T * k + (T if ex.shared is not None else 0)
    y, err = np.full((rows, ex.H), np.nan), np.zeros((rows, ex.H))
    for e in range(ex.E):
        t, i = np.nonzero(idx == e)
        if len(t) and (mask is None or mask[e]):
            y[t * k + i], err[t * k + i] = fp8kit.feed_forward(xq[t], ex.parts[e])
    if ex.shared is not None:
        y[T * k:], err[T * k:] = fp8kit.feed_forward(xq, ex.parts[ex.E])
    return y, err


def hidden(seed, T, H):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g)
    x[:, ::37] *= 10
    return x.to(torch.bfloat16)


def run_experts(ex, x, idx, mask=None, stream=None):
    T, k = idx.shape
    rows = T * k + (T if ex.shared is not None else 0)
    y = torch.full((rows + 1, ex.H), 5.0, device="cuda")
    need = L.moe_fp8_expert_ffn_workspace_bytes(T, ex.H, ex.I, ex.E, k, ex.shared is not None)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    L.moe_fp8_expert_ffn(x.cuda(), T, ex.H, ex.I, ex.E, dev(idx), k, ex.table, ex.shared,
                         None if mask is None else dev(mask), y, ws, need, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert (y[rows] == 5.0).all() and (ws[need:] == 0xFF).all()
    return y[:rows].double().cpu().numpy()


def run_combine(ex, x, idx, w):
    T, k = idx.shape
    out = torch.full((T + 1, ex.H), 5.0, dtype=torch.bfloat16, device="cuda")
    need = L.moe_fp8_expert_ffn_workspace_bytes(T, ex.H, ex.I, ex.E, k, ex.shared is not None)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    L.moe_fp8_expert_ffn_combine(x.cuda(), T, ex.H, ex.I, ex.E, dev(idx), dev(w.astype(np.float32)), k, ex.table,
                                 ex.shared, out, ws, need, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert (out[T] == 5.0).all() and (ws[need:] == 0xFF).all()
    return out[:T].double().cpu().numpy()


def check_experts(ex, T, k, seed, busy=0):
    rng = np.random.default_rng(seed)
    x, idx = hidden(seed, T, ex.H), routing(rng, T, ex.E, k, busy)
    y, err = reference(ex, x.double().numpy(), idx)
    got = run_experts(ex, x, idx)
    assert (np.abs(got - y) <= err + 2.0 ** -24 * np.abs(y)).all()
    w = rng.random((T, k)).astype(np.float32).astype(np.float64)
    want = (w[:, :, None] * y[:T * k].reshape(T, k, -1)).sum(1)
    mag = (w[:, :, None] * (np.abs(y) + err)[:T * k].reshape(T, k, -1)).sum(1)
    off = (w[:, :, None] * err[:T * k].reshape(T, k, -1)).sum(1)
    if ex.shared is not None:
        want, mag, off = want + y[T * k:], mag + np.abs(y[T * k:]) + err[T * k:], off + err[T * k:]
    off = off + (k + 2) * 2.0 ** -24 * mag  # the combine's fused adds
    out = run_combine(ex, x, idx, w)
    assert (np.abs(out - want) <= off + 2.0 ** -8 * (np.abs(want) + off)).all()


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("H,I,E,k", [(256, 128, 16, 2), (160, 96, 5, 5), (512, 416, 12, 3)])
def test_experts(H, I, E, k, shared):
    ex = Experts(H + I, H, I, E, shared)
    for T in (1, 2, 5, 17, 64, 103, 170, 300):
        check_experts(ex, T, k, T)
    check_experts(ex, 90, k, 3, busy=70)    # one expert with many tokens
    check_experts(ex, 260, k, 4, busy=260)


def test_experts_mask_and_bad_numbers():
    """Masked experts' slabs are not read and their rows stay; numbers outside 0 .. E-1 are left out."""
    H, I, E, k = 256, 160, 8, 3
    ex = Experts(5, H, I, E, True)
    rng = np.random.default_rng(2)
    mask = np.array([1, 0, 1, 1, 0, 0, 1, 1], np.uint8)
    for e in np.nonzero(mask == 0)[0]:
        ex.table[e] = 0
    for T in (1, 6, 40, 180, 250):
        x, idx = hidden(T, T, H), routing(rng, T, E, k)
        y, err = reference(ex, x.double().numpy(), idx, mask)
        got = run_experts(ex, x, idx, mask)
        off = np.isnan(y).any(1)
        assert off.any() or T == 1
        assert (got[off] == 5.0).all()
        assert (np.abs(got - y) <= err + 2.0 ** -24 * np.abs(y))[~off].all()
    T = 12
    x, idx = hidden(3, T, H), routing(rng, T, E, k)
    idx = np.where(mask[idx] == 0, 0, idx).astype(np.int32)
    bad = idx.copy()
    bad[3, 1], bad[7, 0] = -1, E
    got, want = run_experts(ex, x, bad), run_experts(ex, x, idx)
    rows = [3 * k + 1, 7 * k]
    assert (got[rows] == 5.0).all()
    keep = np.setdiff1d(np.arange(len(got)), rows)
    assert np.array_equal(got[keep], want[keep])


def test_experts_repeat_and_capture():
    """The same call twice gives the same bits; captured and replayed between eager calls, on two streams at once."""
    ex = Experts(9, 384, 256, 16, True)
    for T in (1, 7, 200):
        rng = np.random.default_rng(T)
        k, H = 4, ex.H
        jobs = []
        need = L.moe_fp8_expert_ffn_workspace_bytes(T, H, ex.I, ex.E, k, 1)
        for i in range(2):
            jobs.append(dict(x=hidden(T + i, T, H).cuda(), idx=dev(routing(rng, T, ex.E, k)),
                             w=dev(rng.random((T, k)).astype(np.float32)),
                             out=torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"),
                             ws=torch.empty(need, dtype=torch.uint8, device="cuda")))

        def call(j, stream=None):
            L.moe_fp8_expert_ffn_combine(j["x"], T, H, ex.I, ex.E, j["idx"], j["w"], k, ex.table, ex.shared, j["out"],
                                         j["ws"], need, torch.cuda.current_stream() if stream is None else stream)
        want = []
        for j in jobs:
            call(j)
            torch.cuda.synchronize()
            want.append(j["out"].clone())
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(3):
            for j in jobs:
                j["out"].zero_()
            torch.cuda.synchronize()
            for j, s in zip(jobs, streams):
                call(j, s)
            torch.cuda.synchronize()
            assert all(torch.equal(j["out"], w) for j, w in zip(jobs, want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for j in jobs:
                call(j)
        for _ in range(3):
            for j in jobs:
                j["out"].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(j["out"], w) for j, w in zip(jobs, want))
            call(jobs[1])
            torch.cuda.synchronize()
