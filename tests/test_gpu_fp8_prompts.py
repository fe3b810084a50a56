"""A layer of FP8 experts on prompts of any length."""
import pytest
import torch

from tests.test_gpu_fp8 import gpu, hidden  # noqa: F401
from tests.test_gpu_fp8_layers import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [4096, 4097, 9000])
def test_more_pairs_than_one_call_takes(T):
    """16384 (token, expert) pairs are one call; the last of several may be a single token."""
    layer = Layer(128, 96, 10, 4, True, 5, 3)
    x = hidden(T, T, layer.H).cuda()
    idx, w = layer.layer.route(x)
    out = layer.layer(x)
    assert out.shape == x.shape
    layer.check(x, idx, w, out)
