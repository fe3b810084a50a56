"""Workspaces that a program keeps: sized for its longest call, they have to do for every shorter one."""
import itertools

import pytest

from routed_expert_streaming_amd import _lib as L

TOKENS = [1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 24, 31, 32, 33, 47, 64, 65, 100, 128, 129, 200, 256, 257, 500, 511, 512, 513,
          700, 1000, 1023, 1024, 1025, 1100, 1500, 2000, 2047, 2048, 2049, 4096, 4097, 5000, 8192, 16384]


@pytest.mark.parametrize("H", [32, 96, 256, 1056, 2048, 6144, 16384])
@pytest.mark.parametrize("E", [1, 8, 64, 96, 128, 160, 256, 1000, 1024])
def test_router(E, H):
    layers = [1, 2, 3, 5, 8, 16, 61, 200, 257]
    size = {(n, T): L.moe_router_scored_workspace_bytes(n, T, E, H) for n in layers for T in TOKENS}
    for (n, T), need in size.items():
        assert need > 0
        for n2, T2 in itertools.product(layers, TOKENS):
            if n2 <= n and T2 <= T:
                assert size[n2, T2] <= need, (n2, T2, n, T)


def test_router_keeps_its_size():
    """The bound is near what the calls take: the split sums of a prompt, or a logit's partial sums of a few tokens."""
    for n, T, E, H in ((1, 2048, 256, 6144), (1, 1024, 256, 6144), (16, 32, 256, 6144), (1, 1, 128, 4096)):
        assert L.moe_router_scored_workspace_bytes(n, T, E, H) <= 1.25 * 4 * E * max(n * T * 32, 32768)


@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("H,I,E,k", [(32, 32, 8, 1), (4096, 1536, 128, 8), (256, 16384, 16, 8), (32, 16384, 4, 4),
                                     (16384, 32, 64, 6), (96, 160, 682, 24), (32, 32, 1024, 16), (64, 64, 1024, 1024),
                                     (1024, 1024, 24, 12), (512, 4096, 40, 40)])
def test_experts(H, I, E, k, shared):
    size = [L.moe_fp8_expert_ffn_workspace_bytes(T, H, I, E, k, shared) for T in range(1, 16384 // k + 1)]
    assert all(a > 0 for a in size) and all(a <= b for a, b in zip(size, size[1:]))
    assert all(a <= L.moe_fp8_expert_ffn_workspace_bytes(T + 1, H, I, E, k, 1) for T, a in enumerate(size[:64]))


@pytest.mark.parametrize("kind", [L.MOE_BF16, L.MOE_FP8])
@pytest.mark.parametrize("N,K", [(16, 16), (4096, 1024), (5000, 640), (20000, 4096), (4096, 50000)])
def test_product(N, K, kind):
    size = [L.moe_fp8_matmul_workspace_bytes(M, N, K, kind) for M in range(1, 600)]
    assert all(a <= b for a, b in zip(size, size[1:]))


def test_router_refuses_more_tokens_than_a_grid_holds():
    how = L.moe_routing(L.MOE_SCORE_SIGMOID, 1, 1, L.MOE_GROUP_MAX, 1, 1.0)
    for T in ((1 << 26) - 3, 1 << 26, (1 << 31) - 1):
        with pytest.raises(L.MoEError) as ei:
            L.moe_router_scored(0x1000, 1, T, 32, 0x1000, None, None, 4, 1, how, 0x1000, 0x1000, 0x1000, 0)
        assert ei.value.status == L.MOE_E_SHAPE
        assert L.moe_router_scored_workspace_bytes(1, T, 4, 32) == 0
    assert L.moe_router_scored_workspace_bytes(1, (1 << 26) - 4, 4, 32) > 0
