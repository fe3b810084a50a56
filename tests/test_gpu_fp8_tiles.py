"""The FP8 product at sizes that reach each of its kernels, in both output types: sums that 32 bits hold exactly have to come
out bit for bit; and matrices whose rows lie so far apart that offsets pass 32 bits."""
import numpy as np
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from tests import fp8kit
from tests.test_gpu_fp8 import DTYPE, dev, gpu, random_operand, run_matmul, small_operand  # noqa: F401

pytestmark = pytest.mark.gpu

# from few rows or columns to tiles of 256 x 256; K of one block to 66 (scales are held 64 blocks at a time), of whole
# blocks and not, of numbers of blocks that groups of 2 and 4 waves do not share evenly
SHAPES = [(4100, 16, 400), (4095, 15, 2080), (1, 8200, 400), (1, 16, 8400), (16, 33, 8400), (33, 8193, 656), (65, 8200, 1040),
          (65, 4101, 8400), (129, 8200, 16), (129, 8200, 144), (130, 8190, 1552), (300, 8199, 400), (300, 12300, 656),
          (1300, 6200, 144), (1299, 6203, 272), (2050, 6149, 144), (1300, 8200, 144), (1311, 8190, 640), (8200, 16, 656),
          (8201, 17, 1552), (513, 516, 16), (16, 8200, 16), (64, 4100, 16)]


@pytest.mark.parametrize("y_type", [L.MOE_BF16, L.MOE_FP32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact(M, N, K, y_type):
    rng = np.random.default_rng(M + N + K)
    a, sa = small_operand(rng, M, K, 1)
    w, sw = small_operand(rng, N, K, 128)
    bias = rng.integers(-50, 51, N).astype(np.float64) if N % 2 else None
    got = run_matmul(a, sa, w, sw, M, N, K, bias, y_type)
    want = fp8kit.values(a, sa, 1) @ fp8kit.values(w, sw, 128).T
    if bias is not None:
        want = want + bias
    assert np.array_equal(got, torch.from_numpy(want).to(DTYPE[y_type]).double().numpy())


@pytest.mark.parametrize("M,N,K", [(130, 8190, 1040), (1299, 6203, 272), (1311, 8190, 400), (65, 4101, 8400)])
def test_bounds(M, N, K):
    rng = np.random.default_rng(M + N)
    a, sa = random_operand(rng, M, K, 1)
    w, sw = random_operand(rng, N, K, 128)
    va, vw = fp8kit.values(a, sa, 1), fp8kit.values(w, sw, 128)
    want, mag = va @ vw.T, np.abs(va) @ np.abs(vw).T
    for y_type, half in ((L.MOE_BF16, 2.0 ** -8), (L.MOE_FP32, 2.0 ** -24)):
        got = run_matmul(a, sa, w, sw, M, N, K, None, y_type)
        err = (fp8kit.sum_error(K) + fp8kit.cores_error(y_type == L.MOE_BF16) + 2.0 ** -24) * mag
        assert (np.abs(got - want) <= err + half * (np.abs(want) + err)).all()


@pytest.mark.parametrize("y_type", [L.MOE_BF16, L.MOE_FP32])
@pytest.mark.parametrize("M,N,K", [(1, 33, 16), (1, 4100, 8400), (2, 257, 4096), (3, 130, 6144), (5, 1000, 2048), (8, 72, 1040),
                                   (11, 8200, 912), (16, 300, 400), (16, 4096, 1024), (16, 4112, 1040), (9, 64, 2064)])
def test_activations_of_a_few_rows(M, N, K, y_type):
    """bf16 activations, quantised in the product's kernel or before it."""
    rng = np.random.default_rng(M * N + K)
    w, sw = random_operand(rng, N, K, 128)
    x = torch.randn((M, K + 8), generator=torch.Generator().manual_seed(K)).to(torch.bfloat16)[:, :K]
    bias = rng.standard_normal(N).astype(np.float32)
    y = torch.full((M + 1, N), 5.0, dtype=DTYPE[y_type], device="cuda")
    need = L.moe_fp8_matmul_workspace_bytes(M, N, K, L.MOE_BF16)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    xd = torch.full((M, K + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    xd[:, :K] = x.cuda()
    L.moe_fp8_matmul(xd, L.MOE_BF16, 2 * (K + 8), None, 0, dev(w), K, dev(sw), 4 * sw.shape[1], M, N, K, dev(bias), y, y_type,
                     N * y.element_size(), ws, need, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert (y[M] == 5.0).all() and (ws[need:] == 0xA5).all()
    va, vw = fp8kit.values(*fp8kit.quantise(x.double().numpy()), 1), fp8kit.values(w, sw, 128)
    want, mag = va @ vw.T + bias, np.abs(va) @ np.abs(vw).T + np.abs(bias)
    err = (fp8kit.sum_error(K) + fp8kit.cores_error(y_type == L.MOE_BF16) + 2.0 ** -24) * mag
    half = 2.0 ** -8 if y_type == L.MOE_BF16 else 2.0 ** -24
    assert (np.abs(y[:M].double().cpu().numpy() - want) <= err + half * (np.abs(want) + err)).all()


def apart(c, stride):
    """Rows of c as a view of rows stride bytes apart."""
    buf = torch.empty(((c.shape[0] - 1) * stride + c.shape[1] * c.element_size(),), dtype=torch.uint8, device="cuda")
    view = buf.view(c.dtype).as_strided(c.shape, (stride // c.element_size(), 1))
    view.copy_(c)
    return view


@pytest.mark.parametrize("M,N,K,far", [(3, 560, 272, "w"), (40, 560, 272, "w"), (560, 40, 272, "a"), (540, 130, 144, "y"),
                                       (1, 560, 400, "w")])
@pytest.mark.parametrize("stride", [(8 << 20) - 16, (8 << 20) + 16])
def test_rows_far_apart(M, N, K, far, stride):
    """Rows up to 4.7 GB behind the first one, on both sides of the distance up to which tiles take them."""
    rng = np.random.default_rng(N)
    a, sa = small_operand(rng, M, K, 1)
    w, sw = small_operand(rng, N, K, 128)
    da, dw = dev(a), dev(w)
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    if far == "a":
        da = apart(da, stride)
    elif far == "w":
        dw = apart(dw, stride)
    else:
        y = apart(y, stride)
    pa = dev(fp8kit.padded(sa))
    need = L.moe_fp8_matmul_workspace_bytes(M, N, K, L.MOE_FP8)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    L.moe_fp8_matmul(da, L.MOE_FP8, da.stride(0), pa, 4 * pa.stride(0), dw, dw.stride(0), dev(sw), 4 * sw.shape[1], M, N, K,
                     None, y, L.MOE_BF16, 2 * y.stride(0), ws, need, torch.cuda.current_stream())
    want = fp8kit.values(a, sa, 1) @ fp8kit.values(w, sw, 128).T
    assert np.array_equal(y.double().cpu().numpy(), torch.from_numpy(want).to(torch.bfloat16).double().numpy())
