"""The product's activation scales as callers may lay them out: rows far apart, and rows that end where their scales do."""
import numpy as np
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from tests import fp8kit
from tests.test_gpu_fp8 import DTYPE, dev, gpu, small_operand  # noqa: F401

pytestmark = pytest.mark.gpu


def product(a, rows, stride, w, sw, y_type):
    """y in float64; rows: the device pointer's tensor of A's scales, stride bytes apart."""
    (M, K), N = a.shape, w.shape[0]
    y = torch.full((M, N), 5.0, dtype=DTYPE[y_type], device="cuda")
    L.moe_fp8_matmul(dev(a), L.MOE_FP8, K, rows, stride, dev(w), K, dev(sw), 4 * sw.shape[1], M, N, K, None, y, y_type,
                     N * y.element_size(), None, 0, torch.cuda.current_stream())
    return y.double().cpu().numpy()


@pytest.mark.parametrize("y_type", [L.MOE_BF16, L.MOE_FP32])
@pytest.mark.parametrize("M,N,K,stride", [(300, 320, 640, (8 << 20) - 16), (300, 4096, 640, (8 << 20) - 16),
                                          (300, 4096, 640, 8 << 20), (300, 4096, 640, (40 << 20) + 64),
                                          (40, 8192, 640, 1 << 28), (16, 64, 144, 1 << 28)])
def test_scale_rows_far_apart(M, N, K, stride, y_type):
    """Up to the 2^28 bytes that the interface names; the gaps hold NaN."""
    rng = np.random.default_rng(M + K)
    a, sa = small_operand(rng, M, K, 1)
    w, sw = small_operand(rng, N, K, 128)
    blocks = fp8kit.blocks(K)
    buf = torch.full(((M - 1) * (stride // 4) + (blocks + 3) // 4 * 4,), float("nan"), device="cuda")
    buf.as_strided((M, blocks), (stride // 4, 1)).copy_(dev(sa))
    got = product(a, buf, stride, w, sw, y_type)
    want = fp8kit.values(a, sa, 1) @ fp8kit.values(w, sw, 128).T
    assert np.array_equal(got, torch.from_numpy(want).to(DTYPE[y_type]).double().numpy())


# one for each kernel that a product may take; blocks of 128 columns that are no multiple of four
ENDS = [(1, 16, 128), (1, 130, 1040), (7, 300, 272), (16, 64, 2080), (17, 130, 144), (33, 260, 640), (17, 5000, 1168),
        (33, 5000, 272), (100, 5000, 784), (33, 5000, 144), (300, 6144, 144), (300, 6144, 1168), (2000, 2080, 144),
        (1500, 6144, 144), (2560, 4864, 144)]


@pytest.mark.parametrize("y_type", [L.MOE_BF16, L.MOE_FP32])
@pytest.mark.parametrize("M,N,K", ENDS)
def test_scale_rows_that_end_with_their_values(M, N, K, y_type):
    """The last row of scales is ceil(K / 128) values and no more; what lies behind it is not the product's."""
    rng = np.random.default_rng(M + N + K)
    a, sa = small_operand(rng, M, K, 1)
    w, sw = small_operand(rng, N, K, 128)
    blocks = fp8kit.blocks(K)
    assert blocks % 4
    row = (blocks + 3) // 4 * 4
    buf = torch.full(((M - 1) * row + blocks,), float("nan"), device="cuda")
    buf.as_strided((M, blocks), (row, 1)).copy_(dev(sa))
    got = torch.from_numpy(product(a, buf, 4 * row, w, sw, y_type))
    va, vw = (dev(fp8kit.values(*o)) for o in ((a, sa, 1), (w, sw, 128)))
    assert torch.equal(got, (va @ vw.T).to(DTYPE[y_type]).double().cpu())  # (sums of whole multiples of 1/4: exact)
