"""Every kernel, tile, part of K and row form of the dense MXFP4 operators that their launch rules can choose."""
import numpy as np
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from tests import mxkit

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


# ------------------------------------------------------------------ product
# (M, N, K, parts of K): 64 x 64 tiles, 128 x 128, 256 x 192 (bf16 128 x 256), the rows kernels.  K past 2048 brings a
# tile's scales in more than once; most last groups of 128 columns, last parts and last tiles are cut short, N is odd,
# even and a multiple of what a 16-byte store holds.
MX_PARTS = [(65, 130, 32800, 8), (98, 1030, 20512, 4), (98, 2168, 8224, 2), (65, 3001, 4128, 1),
            (98, 2168, 32800, 8), (200, 2169, 12320, 4), (520, 1801, 8224, 2), (520, 1801, 4128, 1),
            (520, 1801, 32800, 8), (1000, 2169, 20512, 4), (1030, 4090, 12320, 2), (2040, 2167, 4128, 1),
            (65, 3000, 4128, 1), (520, 1800, 4128, 1), (2040, 2168, 4128, 1), (40, 33, 6176, 1),
            (32, 6001, 1056, 1), (16, 5000, 6176, 1), (8, 4100, 6176, 1)]
BF16_PARTS = [(65, 130, 32800, 8), (65, 130, 6176, 4), (98, 2169, 4128, 2), (40, 4100, 2080, 1),
              (1500, 131, 32800, 8), (65, 5000, 6176, 4), (520, 1801, 4128, 2), (2040, 1030, 4128, 1),
              (257, 1801, 32800, 8), (200, 5000, 12320, 4), (385, 5000, 12320, 2), (2040, 2169, 4128, 1),
              (40, 4104, 2080, 1), (2040, 1032, 4128, 1), (2040, 2168, 4128, 1), (40, 33, 2080, 1),
              (32, 6001, 544, 1), (16, 5000, 6176, 1), (3, 4099, 6176, 1)]


def exact_operands(kind, M, N, K, seed):
    """(a, its values, w, its values, bias, unit of a product).  Scale bytes are drawn per block on both sides (125 ..
    129, for the longest rows 126 .. 128), so that a scale of another block, row or run is seen."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    low, high = (125, 129) if K < 16384 else (126, 128)

    def rows(R):
        codes = torch.randint(0, 16, (R, K), generator=g, device="cuda", dtype=torch.uint8)
        scales = torch.randint(low, high + 1, (R, K // 32), generator=g, device="cuda", dtype=torch.uint8)
        packed = torch.zeros((R, mxkit.row_bytes(K)), dtype=torch.uint8, device="cuda")
        packed[:, :K // 2] = codes[:, 0::2] + 16 * codes[:, 1::2]
        packed[:, K // 2:K // 2 + K // 32] = scales
        e2m1 = torch.tensor([*mxkit.MAGNITUDES, *-mxkit.MAGNITUDES], device="cuda")
        v = e2m1[codes.int()].view(R, -1, 32) * torch.exp2(scales.double() - 127).unsqueeze(-1)
        v = v.reshape(R, K)
        few = slice(0, 2)
        assert np.array_equal(v[few].cpu().numpy(), mxkit.values(codes[few].cpu().numpy().astype(np.int64),
                                                                 scales[few].cpu().numpy().astype(np.int64)))
        return packed, v
    w, wv = rows(N)
    if kind == L.MOE_MXFP4:
        a, av = rows(M)
    else:
        av = torch.randint(-16, 17, (M, K), generator=g, device="cuda").double() * 0.25
        a = av.to(torch.bfloat16)
    b = torch.randint(-64, 65, (N,), generator=g, device="cuda").float()
    least = 0.5 * 2.0 ** (low - 127)  # a weight's unit, and an MXFP4 activation's
    return a, av, w, wv, b, least * (least if kind == L.MOE_MXFP4 else 0.25)


@pytest.mark.parametrize("kind,M,N,K,parts", [(L.MOE_MXFP4, *s) for s in MX_PARTS] +
                         [(L.MOE_BF16, *s) for s in BF16_PARTS])
def test_matmul_exact_sums_in_parts(kind, M, N, K, parts):
    """Every product is a multiple of one unit, and the magnitudes of a result's terms add up to less than 2^24 of
    them (checked on the values themselves): 32 bits hold every partial sum, so every order gives what 64 bits do."""
    a, av, w, wv, b, unit = exact_operands(kind, M, N, K, M + N + K)
    assert float((av.abs() @ wv.abs().t()).max()) + 64 < 2.0 ** 24 * unit
    a_stride, w_stride = a.stride(0) * a.element_size(), w.stride(0)
    need = L.moe_mx_matmul_workspace_bytes(M, N, K, kind)
    assert need == (0 if parts == 1 else 4 * parts * M * N)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN sums
    plain = av @ wv.t()
    for bias in (b, None):
        want = plain + (0.0 if bias is None else bias.double())
        for y_type, dtype in ((L.MOE_FP32, torch.float32), (L.MOE_BF16, torch.bfloat16)):
            for pitch in (N + 5, (N + 7) // 8 * 8):  # rows of y off 16-byte boundaries, and on them
                y = torch.full((M + 1, pitch), 5.0, dtype=dtype, device="cuda")
                L.moe_mx_matmul(a, kind, a_stride, w, w_stride, M, N, K, bias, y, y_type, pitch * y.element_size(), ws,
                                need, torch.cuda.current_stream())
                assert torch.equal(y[:M, :N], want.float().to(dtype)), (y_type, bias is None, pitch)
                y[:M, :N] = 5.0
                assert (y == 5.0).all() and (ws[need:] == 0xFF).all()
    if need:
        with pytest.raises(L.MoEError) as ei:
            L.moe_mx_matmul(a, kind, a_stride, w, w_stride, M, N, K, None, y, L.MOE_BF16, 2 * y.stride(0), ws, need - 1,
                            torch.cuda.current_stream())
        assert ei.value.status == L.MOE_E_NOMEM and (y == 5.0).all()


@pytest.mark.parametrize("kind", [L.MOE_MXFP4, L.MOE_BF16])
@pytest.mark.parametrize("M", [1, 5, 20, 40, 150, 300])
def test_matmul_keeps_subnormal_sums(M, kind):
    """Results in and around fp32's subnormal range: every product is a multiple of 2^-137 and the magnitudes of a
    result's terms stay below 2^-113, so 32 bits hold the sums unless something flushes them to zero."""
    rng = np.random.default_rng(M)
    K, N = 288, 40
    c, s = mxkit.random_rows(rng, N, K, 60, 60)
    w, wv = torch.from_numpy(mxkit.pack(c, s)).cuda(), mxkit.values(c, s)
    if kind == L.MOE_MXFP4:
        c, s = mxkit.random_rows(rng, M, K, 60, 60)
        a, av = torch.from_numpy(mxkit.pack(c, s)).cuda(), mxkit.values(c, s)
    else:
        av = rng.integers(-16, 17, (M, K)) * 0.25 * 2.0 ** -67
        a = torch.from_numpy(av).cuda().to(torch.bfloat16)
    want = av @ wv.T
    assert (np.abs(av) @ np.abs(wv).T).max() < 2.0 ** -113  # 24 bits of the unit
    assert ((want != 0) & (np.abs(want) < 2.0 ** -126)).any()
    y = torch.zeros((M, N), device="cuda")
    need = L.moe_mx_matmul_workspace_bytes(M, N, K, kind)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    L.moe_mx_matmul(a, kind, a.stride(0) * a.element_size(), w, mxkit.row_bytes(K), M, N, K, None, y, L.MOE_FP32, 4 * N,
                    ws, need, torch.cuda.current_stream())
    assert np.array_equal(y.double().cpu().numpy(), want)


# ------------------------------------------------------------------ norms around a block
def norm_roundings(T, H, wide):
    """Roundings on the way to a row's factor and through it: a thread's squares, one after the other (eight values, or
    one, at a time: one time for few rows, two from 256 on, up to four, or as often as 1024 threads need for a
    row beyond that), 6 sums of a wave, the waves' sums, mean, eps, root, reciprocal and three products."""
    V = 8 if wide else 1
    units = -(-H // V)
    items = 1 if T < 256 else 2
    while items < 4 and units > items * 1024:
        items *= 2
    threads = min(-(-(-(-units // items)) // 64) * 64, 1024)
    return V * -(-units // threads) + 6 + threads // 64 - 1 + 7


def offset(t, elements):
    """t's values from `elements` elements into a fresh buffer on."""
    flat = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)
    flat[elements:] = t.flatten()
    return flat[elements:].view(t.shape)


def rms(v, w, eps):
    x = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    return x if w is None else x * w


# rows in registers (one, two, four values or eights of them a thread) and rows read again; streams below and from 4
# MiB on, which are written past the caches; widths and pointers that 16-byte accesses cannot take
@pytest.mark.parametrize("rt", [L.MOE_FP32, L.MOE_BF16])
@pytest.mark.parametrize("T,H,shift", [(3, 1001, 0), (300, 1001, 0), (2, 3001, 0), (3, 5001, 0), (3, 5000, 1),
                                       (2, 6144, 0), (257, 2048, 0), (3, 20000, 0), (3, 40000, 0),
                                       (200, 6144, 0), (600, 6144, 0), (70, 20000, 0), (120, 20000, 0),
                                       (40, 40000, 0), (80, 40000, 0), (2048, 6143, 0)])
def test_block_norm_on_every_path(T, H, shift, rt):
    g = torch.Generator(device="cuda").manual_seed(T * 7 + H)
    dtype = torch.float32 if rt == L.MOE_FP32 else torch.bfloat16
    eps, scale = 1e-6, 0.37

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    add = offset((normal(T, H) * 3).to(torch.bfloat16), shift)
    resid = offset((normal(T, H) * 5).to(dtype), shift)
    w_post, w_pre = 1 + 0.3 * normal(H), 1 + 0.3 * normal(H)
    gate = offset(normal(T, H).to(torch.bfloat16), shift)
    wide = H % 8 == 0 and not shift
    u = norm_roundings(T, H, wide) * 2.0 ** -24
    s = torch.cuda.current_stream()

    def call(resid, out, x, rows):
        L.moe_block_norm(add, 1, w_post, gate, L.MOE_GATE_ELEMENT, scale, resid, out, rt, w_pre, T, H, eps, x, rows, s)
    out, x = torch.full((T + 1, H), 3.0, dtype=dtype, device="cuda"), torch.full((T + 1, H), 3.0, dtype=torch.bfloat16,
                                                                                 device="cuda")
    rows = None
    if wide:
        rows = torch.full((T + 1, mxkit.row_bytes(H)), 0xA5, dtype=torch.uint8, device="cuda")
    before = resid.clone()
    call(resid, out, x, rows)
    assert torch.equal(resid, before) and (out[T] == 3.0).all() and (x[T] == 3.0).all()
    d = rms(add.double(), w_post.double(), eps) * gate.double() * float(np.float32(scale))
    want = before.double() + d
    tol = u * d.abs() + 2.0 ** -24 * want.abs()
    if rt == L.MOE_BF16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert ((out[:T].double() - want).abs() <= tol).all()
    nx = rms(out[:T].double(), w_pre.double(), eps)
    assert ((x[:T].double() - nx).abs() <= (2.0 ** -8 * (1 + u) + u) * nx.abs()).all()
    if wide:
        packed = torch.empty_like(rows[:T])
        L.moe_mx_quant(x, L.MOE_BF16, 2 * H, T, H, L.MOE_MX_SCALE_FLOOR, packed, mxkit.row_bytes(H), None, s)
        assert torch.equal(rows[:T], packed) and (rows[T] == 0xA5).all()
        rows.fill_(0xA5)
        call(resid, out, None, rows)  # the rows alone
        assert torch.equal(rows[:T], packed) and (rows[T] == 0xA5).all()
    # in place, with and without a next block: the same bits
    for follow in (x.clone(), None):
        inplace = offset(before, shift)
        call(inplace, inplace, follow, None)
        assert torch.equal(inplace, out[:T]) and (follow is None or torch.equal(follow, x))
    # the pre-norm of the kept stream alone
    alone = torch.full_like(x, 3.0)
    L.moe_block_norm(None, 0, None, None, L.MOE_GATE_NONE, scale, inplace, None, rt, w_pre, T, H, eps, alone, None, s)
    assert torch.equal(alone, x)


# ------------------------------------------------------------------ more rows than one launch takes, and one row
def test_quant_in_two_launches():
    """2^28 rows of 32 columns are 2^30 lanes, the most of one launch: five rows more."""
    rows, K = (1 << 28) + 5, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    edge = [0, 1, (1 << 28) - 1, 1 << 28, rows - 1]
    x[edge] = torch.randn((len(edge), K), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((rows, 32), 0xA5, dtype=torch.uint8, device="cuda")
    vals = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    L.moe_mx_quant(x, L.MOE_BF16, 2 * K, rows, K, L.MOE_MX_SCALE_FLOOR, out, 32, vals, torch.cuda.current_stream())
    codes, scales = mxkit.quantise(x[edge].double().cpu().numpy(), "floor")
    assert np.array_equal(out[edge].cpu().numpy(), mxkit.pack(codes, scales))
    assert np.array_equal(vals[edge].double().cpu().numpy(), mxkit.values(codes, scales))
    ones = out[2].clone()  # a row of ones; every other row but the edge ones is one
    assert ones[16] == 125 and (ones[:16] == 0x66).all()
    same = (out.view(torch.int64) == ones.view(torch.int64)).all(1)
    assert int(same.sum()) == rows - len(edge) and (vals[2:1000] == 1.0).all() and (vals[-4:-1] == 1.0).all()


@pytest.mark.parametrize("kind", [L.MOE_GATE_ROW, L.MOE_GATE_ELEMENT])
def test_block_norm_in_two_launches(kind):
    """2^20 rows are the most of one launch: the others, on every operand, against a call on those rows alone."""
    T, H = (1 << 20) + 37, 32
    g = torch.Generator(device="cuda").manual_seed(2)
    add = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    resid = torch.randn((T, H), generator=g, device="cuda")
    gate = torch.rand((T,) if kind == L.MOE_GATE_ROW else (T, H), generator=g, device="cuda")
    gate = gate if kind == L.MOE_GATE_ROW else gate.to(torch.bfloat16)

    def call(lo, hi):
        n = hi - lo
        out, x = torch.empty((n, H), device="cuda"), torch.empty((n, H), dtype=torch.bfloat16, device="cuda")
        rows = torch.empty((n, mxkit.row_bytes(H)), dtype=torch.uint8, device="cuda")
        L.moe_block_norm(add[lo:hi], 1, None, gate[lo:hi], kind, 0.5, resid[lo:hi], out, L.MOE_FP32, None, n, H, 1e-6,
                         x, rows, torch.cuda.current_stream())
        return out, x, rows
    whole = call(0, T)
    for lo, hi in ((0, 8), ((1 << 20) - 8, 1 << 20), (1 << 20, T)):
        for a, b in zip(whole, call(lo, hi)):
            assert torch.equal(a[lo:hi], b)


@pytest.mark.parametrize("kind", [L.MOE_MXFP4, L.MOE_BF16])
def test_matmul_rows_in_two_launches(kind):
    """Rows of W far apart take the rows kernel at any M, a grid of which holds 65535 tiles of 32 rows."""
    M, N, K, apart = 65535 * 32 + 41, 3, 64, 9 << 20
    g = torch.Generator(device="cuda").manual_seed(3)
    packed = torch.zeros((N, mxkit.row_bytes(K)), dtype=torch.uint8, device="cuda")
    packed[:, :K // 2] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    packed[:, K // 2:K // 2 + K // 32] = 127
    w = torch.zeros((N, apart), dtype=torch.uint8, device="cuda")
    w[:, :packed.shape[1]] = packed
    if kind == L.MOE_MXFP4:
        a = torch.zeros((M, mxkit.row_bytes(K)), dtype=torch.uint8, device="cuda")
        a[:, :K // 2] = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        a[:, K // 2:K // 2 + K // 32] = 126
    else:
        a = torch.randint(-16, 17, (M, K), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.full((M + 1, N), 5.0, device="cuda")
    L.moe_mx_matmul(a, kind, a.stride(0) * a.element_size(), w, apart, M, N, K, None, y, L.MOE_FP32, 4 * N, None, 0,
                    torch.cuda.current_stream())
    assert (y[M] == 5.0).all()

    def values(rows):
        r = rows.cpu().numpy()
        codes = np.stack([r[:, :K // 2] & 15, r[:, :K // 2] >> 4], -1).reshape(len(r), K).astype(np.int64)
        return mxkit.values(codes, r[:, K // 2:K // 2 + K // 32].astype(np.int64))
    for lo, hi in ((0, 70), (65535 * 32 - 35, 65535 * 32 + 35), (M - 35, M)):
        av = values(a[lo:hi]) if kind == L.MOE_MXFP4 else a[lo:hi].double().cpu().numpy()
        assert np.array_equal(y[lo:hi].double().cpu().numpy(), av @ values(packed).T)


@pytest.mark.parametrize("kind", [L.MOE_MXFP4, L.MOE_BF16])
def test_strides_of_one_row_are_not_read(kind):
    K, odd = 288, -7
    a, av, w, wv, _, _ = exact_operands(kind, 1, 1, K, 5)
    y = torch.zeros(2, device="cuda")
    L.moe_mx_matmul(a, kind, odd, w, odd, 1, 1, K, None, y, L.MOE_FP32, odd, None, 0, torch.cuda.current_stream())
    assert float(y[0]) == float(av @ wv.t()) and float(y[1]) == 0.0
    if kind == L.MOE_BF16:
        out = torch.zeros(mxkit.row_bytes(K), dtype=torch.uint8, device="cuda")
        L.moe_mx_quant(a, kind, odd, 1, K, L.MOE_MX_SCALE_FIT, out, odd, None, torch.cuda.current_stream())
        assert np.array_equal(out.cpu().numpy(), mxkit.pack(*mxkit.quantise(av.cpu().numpy(), "fit"))[0])


@pytest.mark.parametrize("H", [64, 63])
def test_block_norm_squares_beyond_fp32(H):
    """What the interface says of rows whose squares leave fp32's range; the rows beside them are as ever."""
    resid = torch.ones((5, H), device="cuda")
    resid[1], resid[2], resid[3] = 1e19, 1e-24, 0.0  # 1e38 * H is beyond fp32, 1e-48 below it
    s = torch.cuda.current_stream()
    for eps in (0.0, 1e-6):
        x = torch.empty((5, H), dtype=torch.bfloat16, device="cuda")
        L.moe_block_norm(None, 0, None, None, L.MOE_GATE_NONE, 1.0, resid, None, L.MOE_FP32, None, 5, H, eps, x, None,
                         s)
        assert (x[0] == 1.0).all() and (x[4] == 1.0).all() and (x[1] == 0.0).all()
        if eps:
            assert ((x[2].float() - 1e-21).abs() <= 1e-21 * 2.0 ** -7).all() and (x[3] == 0.0).all()
        else:
            assert x[2].isinf().all() and x[3].isnan().all()
