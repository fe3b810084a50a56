"""Routing by scores where the logits' sums decide: experts that differ in the last bits, numbers of tokens around those
where another kernel sums, values whose products pass 32 bits' range."""
import numpy as np
import pytest
import torch

from tests import fp8kit
from tests.test_gpu_router_scored import Call, check, gpu, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [1, 5, 8, 9, 16, 17, 31, 32, 33, 64, 65])
def test_tokens(T, score):
    for layers in (1, 2):
        x, w, b, c = inputs(T, layers, T, 544, 96, True, True)
        args = (6, score, 8, 3, "top2", True, 2.5)
        check(Call(x, w, b, c, *args), x, w, b, c, *args)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,H", [(6, 256, 1024), (70, 256, 1024), (40, 640, 96), (300, 64, 2080)])
def test_experts_that_differ_in_the_last_bits(T, E, H, score):
    """Runs of 16 experts whose router rows are the same but for a few last bits, scattered: their logits round to the same
    or to neighbouring 32-bit values, and which is decided by the 64-bit sum."""
    rng = np.random.default_rng(E)
    x, w, _, _ = inputs(E + T, 1, T, H, E, False)
    base = w[0, rng.permutation(E)[:E // 16]]
    rows = np.repeat(base, 16, axis=0).astype(np.float32)
    at = rng.integers(0, H, (E, 3))
    for e in range(E):
        for h in at[e]:
            rows[e, h] = np.nextafter(rows[e, h], np.float32(rng.choice([-9, 9])))
    w = rows[rng.permutation(E)][None].astype(np.float64)
    for args in ((12, score, 1, 1, "max", True, 1.0), (8, score, 4, 2, "top2", False, 1.0)):
        check(Call(x, w, None, None, *args), x, w, None, None, *args)


@pytest.mark.parametrize("T", [3, 50])
@pytest.mark.parametrize("size", [(1e19, 1e17), (1e30, 1e7), (1e-30, 1e-10), (1e38, 1e-38)])
def test_large_and_small_values(T, size):
    """Logits up to 1e38 and down to subnormal ones; norms beyond 32 bits.  Experts only: a score of such logits is 0, 1 or
    one half."""
    x, w, _, c = inputs(3, 1, T, 160, 48, True)
    x = torch.from_numpy(x * size[0]).to(torch.bfloat16).double().numpy()
    w = (w * size[1]).astype(np.float32).astype(np.float64)
    rows = np.isfinite(x[0]).all(1)  # inputs have to be finite: 1e38 times what is above 3.39 (four of 8000) is not in bf16
    for balance in (None, c):
        for args in ((5, "sigmoid", 1, 1, "max", True, 1.0), (5, "softmax", 4, 2, "max", True, 1.0)):
            idx, wt = Call(x, w, None, balance, *args).run().result()
            ri, _ = fp8kit.route(fp8kit.logits(x[0, rows], w[0], None), None if balance is None else balance[0], *args)
            assert np.array_equal(idx[0, rows], ri) and np.isfinite(wt[0, rows]).all()


@pytest.mark.parametrize("T", [3, 50])
@pytest.mark.parametrize("size", [(1e30, 1e-25), (1e-25, 1e25), (1e36, 1e-37), (1e37, 1e-44)])
def test_squares_that_vanish(T, size):
    """Rows whose squares are below 32 bits' range while their products with the other operand are not; weights with bits
    below bf16's range."""
    x, w, _, c = inputs(13, 1, T, 160, 48, True)
    x = torch.from_numpy(x * size[0]).to(torch.bfloat16).double().numpy()
    w = (w * size[1]).astype(np.float32).astype(np.float64)
    for balance in (None, c):
        for args in ((5, "sigmoid", 1, 1, "max", True, 1.0), (5, "softmax", 4, 2, "max", True, 1.0)):
            idx, wt = Call(x, w, None, balance, *args).run().result()
            ri, rw = fp8kit.route(fp8kit.logits(x[0], w[0], None), None if balance is None else balance[0], *args)
            assert np.array_equal(idx[0], ri) and np.isfinite(wt).all()
