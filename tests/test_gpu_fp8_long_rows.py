"""FP8 experts and products whose rows are more than 64 blocks of 128 columns: a wave holds the scales of 64 blocks and
loads the next ones on the way."""
import numpy as np
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from tests.test_gpu_fp8 import Experts, check_experts, gpu, run_matmul, small_operand  # noqa: F401
from tests.test_gpu_fp8 import DTYPE
from tests import fp8kit

pytestmark = pytest.mark.gpu


# gate/up walks H, down I; the last block of 8192 + 32 columns is cut short, those of 8192 and 8320 are whole
@pytest.mark.parametrize("H,I", [(8192, 32), (8224, 32), (8320, 64), (16384, 32), (16352, 32), (32, 8192), (32, 8224),
                                 (64, 8320), (32, 16384), (32, 16352)])
def test_experts_of_long_rows(H, I):
    E, k = 3, 2
    ex = Experts(H + I, H, I, E, True)
    # a few tokens; tiles of 16 rows (below 24 pairs an expert), of 64 (below 64) and of up to 160
    for T in (2, 9, 50, 130):
        check_experts(ex, T, k, T)


@pytest.mark.parametrize("y_type", [L.MOE_BF16, L.MOE_FP32])
@pytest.mark.parametrize("M,N,K", [(1, 40, 8192), (16, 40, 8224), (20, 72, 8336), (40, 8192, 8320), (60, 4100, 16400),
                                   (300, 4096, 8208), (300, 6144, 8336), (1500, 6144, 8320), (2560, 4864, 8208)])
def test_products_of_long_rows(M, N, K, y_type):
    """Whole numbers up to 8 with scales of one half to two: terms are quarters up to 256 and their sums, of either sign,
    stay far below the 2^22 up to which 32 bits hold quarters."""
    rng = np.random.default_rng(M + N + K)
    (a, sa), (w, sw) = small_operand(rng, M, K, 1), small_operand(rng, N, K, 128)
    got = run_matmul(a, sa, w, sw, M, N, K, None, y_type)
    va, vw = (torch.from_numpy(fp8kit.values(*o)).cuda() for o in ((a, sa, 1), (w, sw, 128)))
    want = (va @ vw.T).to(DTYPE[y_type]).double().cpu().numpy()
    assert np.array_equal(got, want)
