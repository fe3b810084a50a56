"""What the matrix cores keep of a sum, where a statement of the library rests on it: the scored router's logits of many
tokens (three bf16 products and a bound on their error, which decides what is summed again) and the FP8 products of bf16
outputs (the bits of eight products down to 2^-13 of the largest)."""
import numpy as np
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from tests import fp8kit
from tests.test_gpu_fp8 import gpu, run_matmul  # noqa: F401
from tests.test_gpu_router_scored import Call

pytestmark = pytest.mark.gpu


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).double().numpy()


def planes(w):
    """w (float32 values) as three bf16 numbers, each cut off the top of what is left."""
    out, left = [], w.astype(np.float32)
    for _ in range(3):
        p = (left.view(np.uint32) & 0xFFFF0000).view(np.float32)
        out.append(p.astype(np.float64))
        left = left - p
    assert (left == 0).all()
    return out


def data(kind, T, H, E, rng):
    """x [T, H] and w [E, H] whose logits are all different and of size one."""
    x, w = 1 + rng.random((T, H)), 1 + rng.random((E, H))
    if kind == "signs":  # sums that nearly cancel
        x *= rng.choice([-1.0, 1.0], (T, H))
    elif kind == "spikes":  # of eight neighbouring columns one product, or one weight, far above the others
        at = rng.integers(0, 8, H // 8) + 8 * np.arange(H // 8)
        x[:, at] *= 512.0
        w[:, at[::2]] *= 16.0
    x = bf16(x)
    norm = np.sqrt((x ** 2).sum(1).mean()) * np.sqrt((w ** 2).sum(1).mean())
    w = (w * (np.linspace(0.5, 1.5, E) / norm)[:, None]).astype(np.float32).astype(np.float64)
    return x, w


def columns(T, H, E):
    """Columns of H that one workgroup sums in 32 bits: as many parts as make a workgroup a CU, at most 16, of at least
    four times 64 columns."""
    tiles, stages = -(-E // 128) * (1 if T <= 32 else -(-T // 128)), -(-H // 64)
    return 64 * -(-stages // max(1, min(256 // tiles, stages // 4, 16)))


@pytest.mark.parametrize("kind", ["same sign", "signs", "spikes"])
@pytest.mark.parametrize("T,H,E", [(40, 512, 48), (40, 6144, 64), (33, 96, 64), (300, 2080, 64), (300, 16384, 32)])
def test_split_logits_are_within_their_bound(T, H, E, kind):
    """All experts are chosen and their sigmoids returned, from which their logits follow to 2^-24 / (1 - p).  A logit is
    off by at most, relative to the norms of its rows of x and w: per 64 columns two sums of 32 products of the large plane
    (12 * 2^-23 together) and four of the small ones on sums below 2^-7 of it (four more units cover them), one addition
    (2^-24) per 64 columns of a part; and the roundings of both logits (2^-24 each).  (Experts whose sigmoids this does not
    tell apart are summed exactly by the library; few are, but of sums that nearly cancel.)  Without its third plane a
    weight is off by up to 2^-16 of itself, on average half of that, which same-signed data adds up beyond the bound."""
    rng = np.random.default_rng(T + H)
    x, w = data(kind, T, H, E, rng)
    want = x @ w.T
    size = np.sqrt((x ** 2).sum(1))[:, None] * np.sqrt((w ** 2).sum(1))[None]
    bound = (16 + (columns(T, H, E) / 64 + 1) / 2) * 2.0 ** -23 * size + 2.0 ** -23 * np.abs(want)
    if kind != "signs":
        apart = np.diff(np.sort(1 / (1 + np.exp(-want)), 1), axis=1) > bound.max()
        assert apart.mean() > 0.98
    if kind == "same sign":  # this data shows a missing plane
        lost = x @ (w - sum(planes(w)[:2])).T
        assert (np.abs(lost) > 1.5 * bound).mean() > 0.9
    idx, p = (a[0] for a in Call(x[None], w[None], None, None, E, "sigmoid", 1, 1, "max", False, 1.0).run().result())
    assert (np.sort(idx, 1) == np.arange(E)).all()
    got, by = np.empty_like(want), np.empty_like(want)
    np.put_along_axis(got, idx, np.log(p / (1 - p)), 1)
    np.put_along_axis(by, idx, p, 1)
    off = np.abs(got - want) - 1.01 * 2.0 ** -24 / (1 - by)
    print(f"{kind} {T} x {H} x {E}: at most {(off / bound).max():.3f} of the bound, {(off / size).max():.2e} of the norms")
    assert (off <= bound).all()


@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (20, 256, 256), (40, 8192, 640), (300, 6144, 256), (1500, 6144, 256),
                                   (2560, 4864, 256)])
def test_fp8_products_keep_what_is_stated(M, N, K):
    """Eight neighbouring columns hold one product of 448 * 448 and seven small ones; the next block takes the large ones
    away again, so that what is left is what was kept of the small ones.  What lies on the grid of 2^-13 of the large
    product's power of two, 2^(17 - 13) = 16, is kept; of what lies between, less than 16 may be lost of each.  With fp32
    outputs, whose products are exact, nothing is."""
    rng = np.random.default_rng(M + N)
    big = 8 * np.arange(16) + rng.integers(0, 8, 16)
    one = np.ones((M, fp8kit.blocks(K)), np.float32), np.ones((fp8kit.blocks(N), fp8kit.blocks(K)), np.float32)
    for small in ([4.0, 8.0], [4.0, 4.5, 5.0, 5.5]):  # products 16, 32 and 64; from 16 to 30.25
        va, vw = rng.choice(small, (M, K)), rng.choice(small, (N, K))
        va[:, 128:], vw[:, 128:] = 0.0, 0.0
        va[:, big], vw[:, big] = 448.0, 448.0
        va[:, 128 + big], vw[:, 128 + big] = 448.0, -448.0
        a, w = ((fp8kit.nearest(np.abs(v)) + 128 * (v < 0)).astype(np.uint8) for v in (va, vw))
        assert np.array_equal(fp8kit.VALUES[a], va) and np.array_equal(fp8kit.VALUES[w], vw)
        want = (torch.from_numpy(va).cuda() @ torch.from_numpy(vw).cuda().T).cpu().numpy()
        assert np.array_equal(run_matmul(a, one[0], w, one[1], M, N, K, None, L.MOE_FP32), want)
        got = run_matmul(a, one[0], w, one[1], M, N, K, None, L.MOE_BF16)
        if len(small) == 2:
            assert np.array_equal(got, torch.from_numpy(want).to(torch.bfloat16).double().numpy())
        else:
            assert (got >= 16 * 7 * 16).all() and (got <= want * (1 + 2.0 ** -8)).all()
