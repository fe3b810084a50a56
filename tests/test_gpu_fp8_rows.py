"""The experts' kernels at the edges of their tiles: every count of rows an expert may have beside one, every length of
their K loops, masks, numbers that are no expert's, an expert named twice; and the permutation at its largest."""
import numpy as np
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from tests import fp8kit
from tests.test_gpu_fp8 import Experts, dev, gpu, hidden, reference, run_experts, routing  # noqa: F401

pytestmark = pytest.mark.gpu

# rows of each expert, one a token; on average fewer than 24, from there to 64, and more
FEW = (0, 1, 15, 16, 17, 33, 48, 5, 0, 2, 31, 32, 0, 0, 3, 7)
SOME = (0, 1, 15, 16, 17, 33, 64, 65, 90, 128, 129, 0, 20)
MANY = (0, 1, 15, 16, 17, 63, 64, 65, 96, 97, 128, 129, 160, 161, 300, 330)


def check(ex, x, idx, mask=None):
    y, err = reference(ex, x.double().numpy(), idx, mask)
    got = run_experts(ex, x, idx, mask)
    off = np.isnan(y).any(1)
    assert (got[off] == 5.0).all()
    assert (np.abs(got - y) <= err + 2.0 ** -24 * np.abs(y))[~off].all()
    return got


def of_counts(rng, counts):
    return rng.permutation(np.repeat(np.arange(len(counts)), counts)).astype(np.int32)[:, None]


@pytest.mark.parametrize("counts", [FEW, SOME, MANY])
@pytest.mark.parametrize("H,I", [(96, 32), (224, 160), (256, 128), (384, 288), (480, 416), (1120, 544)])
def test_rows_and_blocks(H, I, counts):
    """H and I of 1 to 9 blocks, the last one whole or not."""
    rng = np.random.default_rng(H)
    ex = Experts(H + I, H, I, len(counts), H == 384)
    check(ex, hidden(I, sum(counts), H), of_counts(rng, counts))


@pytest.mark.parametrize("counts", [FEW, SOME, MANY])
def test_masks_and_bad_numbers(counts):
    rng = np.random.default_rng(1)
    E = len(counts)
    ex = Experts(3, 160, 96, E, True)
    mask = (np.arange(E) % 3 != 1).astype(np.uint8)
    for e in np.nonzero(mask == 0)[0]:
        ex.table[e] = 0
    idx = of_counts(rng, counts)
    idx[::11] = np.array([-1, E, 1 << 30, -(1 << 31)])[np.arange(len(idx[::11])) % 4][:, None]
    check(ex, hidden(4, len(idx), 160), idx, mask)
    check(ex, hidden(4, len(idx), 160), idx, np.zeros(E, np.uint8))  # the shared expert alone
    check(ex, hidden(4, len(idx), 160), np.full_like(idx, E), mask)


@pytest.mark.parametrize("T", [1, 3, 4, 40, 400])
def test_an_expert_named_twice(T):
    rng = np.random.default_rng(T)
    ex = Experts(8, 256, 160, 6, True)
    idx = routing(rng, T, 6, 3)
    idx[:, 2] = idx[:, 0]
    idx[::2, 1] = idx[::2, 0]
    got = check(ex, hidden(T, T, 256), idx)
    assert np.array_equal(got[0:3 * T:3], got[2:3 * T:3])


@pytest.mark.parametrize("T,k", [(1, 8), (1, 32), (2, 16), (4, 8), (4, 9), (5, 6), (3, 1), (4, 1)])
def test_few_tokens(T, k):
    """Both sides of the rule for a few tokens, with all tokens of an expert and none."""
    ex = Experts(T + k, 512, 288, 36, T % 2 == 0)
    rng = np.random.default_rng(k)
    check(ex, hidden(T, T, 512), routing(rng, T, 36, k))
    check(ex, hidden(T, T, 512), np.tile(routing(rng, 1, 36, k), (T, 1)))


@pytest.mark.parametrize("T,k,E", [(16384, 1, 1024), (2048, 8, 1024), (16384, 1, 1), (4096, 4, 5)])
def test_the_most_pairs(T, k, E):
    rng = np.random.default_rng(T)
    ex = Experts(6, 32, 32, E, False)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    if E == 1024:
        idx[idx % 7 == 3] = 500  # some experts with none, one with thousands
    check(ex, hidden(T, T, 32), idx)


@pytest.mark.parametrize("T", [2, 90, 700])
def test_values_that_are_not_numbers(T):
    """An infinity in a token's x makes that token's rows NaN and no others; so does a NaN code of an expert's weights,
    in every row of the expert."""
    ex = Experts(12, 224, 96, 6, False)
    rng = np.random.default_rng(T)
    idx = routing(rng, T, 6, 2)
    x = hidden(T, T, 224)
    clean = run_experts(ex, x, idx)
    x[T - 1, 200] = float("inf")
    got = run_experts(ex, x, idx)
    assert np.isnan(got[2 * T - 2:]).all() and np.array_equal(got[:2 * T - 2], clean[:2 * T - 2])
    ex.pool.view(-1)[int(ex.table[2].item()) - ex.pool.data_ptr() + 2 * 224 * 96 + 95] = 0x7F  # W2 row 0, its last column
    got = run_experts(ex, x, idx)
    hit = (idx == 2).reshape(-1)
    hit[2 * T - 2:] = False
    assert np.isnan(got[hit, 0]).all()
    keep = ~hit
    keep[2 * T - 2:] = False
    assert np.array_equal(got[keep], clean[keep]) and np.array_equal(got[hit, 1:], clean[hit, 1:])
