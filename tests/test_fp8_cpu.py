"""Routing by scores and the FP8 operators without a GPU: their refusals, and the numpy forms the GPU tests compare with."""
import numpy as np
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from tests import fp8kit

FAKE = 0x1000  # never dereferenced: the calls below fail validation or have nothing to do
ODD = FAKE + 2


def status(fn, *args):
    with pytest.raises(L.MoEError) as ei:
        fn(*args)
    return ei.value.status


def test_router_refusals():
    def r(x=FAKE, layers=1, T=4, H=64, w=FAKE, bias=None, balance=None, E=16, k=2, score=0, groups=1, top=1, rule=0,
          renorm=1, scale=1.0, how=True, idx=FAKE, wt=FAKE, ws=FAKE, space=1 << 20):
        how = L.moe_routing(score, groups, top, rule, renorm, scale) if how else None
        return status(L.moe_router_scored, x, layers, T, H, w, bias, balance, E, k, how, idx, wt, ws, space)
    assert r(T=-1) == L.MOE_E_ARG and r(layers=-1) == L.MOE_E_ARG and r(how=False) == L.MOE_E_ARG
    assert r(score=2) == L.MOE_E_ARG and r(score=-1) == L.MOE_E_ARG
    assert r(rule=2) == L.MOE_E_ARG and r(rule=-1) == L.MOE_E_ARG
    for scale in (float("nan"), float("inf")):
        assert r(scale=scale) == L.MOE_E_ARG
    for H in (0, -32, 48, 16416):
        assert r(H=H) == L.MOE_E_SHAPE
    for E in (0, -1, 1025):
        assert r(E=E) == L.MOE_E_SHAPE
    for k in (0, -1, 17, 65):
        assert r(k=k) == L.MOE_E_SHAPE
    assert r(groups=0) == L.MOE_E_SHAPE and r(groups=3) == L.MOE_E_SHAPE and r(E=130, groups=65, top=65) == L.MOE_E_SHAPE
    assert r(groups=4, top=0) == L.MOE_E_SHAPE and r(groups=4, top=5) == L.MOE_E_SHAPE
    assert r(groups=4, top=2, k=9) == L.MOE_E_SHAPE  # two groups of four experts
    assert r(groups=16, top=4, rule=1) == L.MOE_E_SHAPE  # two scores of groups of one
    for name in ("x", "w", "idx", "wt", "ws"):
        assert r(**{name: None}) == L.MOE_E_ARG
    assert r(x=ODD) == L.MOE_E_ARG and r(w=ODD) == L.MOE_E_ARG and r(ws=ODD) == L.MOE_E_ARG
    need = L.moe_router_scored_workspace_bytes(2, 4, 16, 64)
    assert need > 0 and r(layers=2, space=need - 1) == L.MOE_E_NOMEM
    assert r(layers=65536, T=1, space=1 << 40) == L.MOE_E_SHAPE
    how = L.moe_routing(0, 1, 1, 0, 0, 1.0)
    L.moe_router_scored(None, 0, 4, 64, None, None, None, 16, 2, how, None, None, None, 0)  # nothing to do
    L.moe_router_scored(None, 2, 0, 64, None, None, None, 16, 2, how, None, None, None, 0)
    for bad in ((0, 4, 16, 64), (1, 0, 16, 64), (1, 4, 0, 64), (1, 4, 1025, 64), (1, 4, 16, 0)):
        assert L.moe_router_scored_workspace_bytes(*bad) == 0


def test_quant_refusals():
    def q(x=FAKE, t=L.MOE_BF16, xs=128, rows=2, K=64, block=1, rule=0, codes=FAKE, cs=64, scales=FAKE, ss=4):
        return status(L.moe_fp8_quant, x, t, xs, rows, K, block, rule, codes, cs, scales, ss)
    assert q(rows=-1) == L.MOE_E_ARG
    assert q(t=L.MOE_MXFP4) == L.MOE_E_ARG and q(t=L.MOE_FP8) == L.MOE_E_ARG and q(t=-1) == L.MOE_E_ARG
    assert q(rule=2) == L.MOE_E_ARG and q(rule=-1) == L.MOE_E_ARG
    for block in (0, 2, 64, 127):
        assert q(block=block) == L.MOE_E_ARG
    for K in (0, -16, 24, (1 << 28) + 16):
        assert q(K=K) == L.MOE_E_SHAPE
    for name in ("x", "codes", "scales"):
        assert q(**{name: None}) == L.MOE_E_ARG
    assert q(xs=112) == L.MOE_E_SHAPE and q(cs=48) == L.MOE_E_SHAPE and q(ss=0) == L.MOE_E_SHAPE
    assert q(xs=-128) == L.MOE_E_SHAPE and q(t=L.MOE_FP32) == L.MOE_E_SHAPE  # 128 bytes hold half a row
    assert q(rows=129, block=128, ss=0) == L.MOE_E_SHAPE  # two rows of blocks
    assert q(x=ODD) == L.MOE_E_ARG and q(codes=ODD) == L.MOE_E_ARG and q(scales=ODD) == L.MOE_E_ARG
    assert q(xs=136) == L.MOE_E_ARG and q(cs=72) == L.MOE_E_ARG and q(ss=6) == L.MOE_E_ARG
    L.moe_fp8_quant(None, L.MOE_BF16, 0, 0, 64, 1, 0, None, 0, None, 0)  # no rows: nothing to do


def test_matmul_refusals():
    def m(a=FAKE, at=L.MOE_FP8, as_=64, sc=FAKE, ss=16, w=FAKE, ws=64, wsc=FAKE, wss=4, M=2, N=2, K=64, bias=None, y=FAKE,
          yt=L.MOE_FP32, ys=8, space=FAKE, n=1 << 20):
        return status(L.moe_fp8_matmul, a, at, as_, sc, ss, w, ws, wsc, wss, M, N, K, bias, y, yt, ys, space, n)
    assert m(M=-1) == L.MOE_E_ARG and m(N=-1) == L.MOE_E_ARG
    assert m(at=L.MOE_FP32) == L.MOE_E_ARG and m(at=L.MOE_MXFP4) == L.MOE_E_ARG and m(at=5) == L.MOE_E_ARG
    assert m(yt=L.MOE_FP16) == L.MOE_E_ARG and m(yt=L.MOE_FP8) == L.MOE_E_ARG
    for K in (0, -64, 40, (1 << 27) + 16):
        assert m(K=K) == L.MOE_E_SHAPE
    for name in ("a", "sc", "w", "wsc", "y"):
        assert m(**{name: None}) == L.MOE_E_ARG
    assert m(as_=48) == L.MOE_E_SHAPE and m(ws=48) == L.MOE_E_SHAPE and m(ys=4) == L.MOE_E_SHAPE
    assert m(ss=0) == L.MOE_E_SHAPE and m(N=129, ys=516, wss=0) == L.MOE_E_SHAPE
    assert m(at=L.MOE_BF16, as_=112) == L.MOE_E_SHAPE
    assert m(a=ODD) == L.MOE_E_ARG and m(w=ODD) == L.MOE_E_ARG and m(sc=FAKE + 4) == L.MOE_E_ARG
    assert m(as_=72) == L.MOE_E_ARG and m(ws=72) == L.MOE_E_ARG and m(ss=20) == L.MOE_E_ARG
    assert m(wsc=ODD) == L.MOE_E_ARG and m(N=129, ys=516, wss=6) == L.MOE_E_ARG
    assert m(y=ODD) == L.MOE_E_ARG and m(ys=10) == L.MOE_E_ARG and m(bias=ODD) == L.MOE_E_ARG
    assert m(M=(1 << 26) + 1) == L.MOE_E_SHAPE and m(N=(1 << 26) + 1, ys=1 << 40) == L.MOE_E_SHAPE
    assert m(as_=(1 << 28) + 16) == L.MOE_E_SHAPE and m(ws=(1 << 28) + 16) == L.MOE_E_SHAPE
    for M, N, K in ((2, 2, 64), (300, 500, 272), (16, 4096, 4096)):
        need = L.moe_fp8_matmul_workspace_bytes(M, N, K, L.MOE_BF16)
        if need:
            assert m(at=L.MOE_BF16, as_=2 * K, M=M, N=N, K=K, ws=K, wss=4096, ys=4 * N, n=need - 1) == L.MOE_E_NOMEM
            assert m(at=L.MOE_BF16, as_=2 * K, M=M, N=N, K=K, ws=K, wss=4096, ys=4 * N, space=None) == L.MOE_E_NOMEM
            assert m(at=L.MOE_BF16, as_=2 * K, M=M, N=N, K=K, ws=K, wss=4096, ys=4 * N, space=ODD) == L.MOE_E_ARG
    for M, N in ((0, 2), (2, 0)):  # nothing to compute
        L.moe_fp8_matmul(None, L.MOE_FP8, 0, None, 0, None, 0, None, 0, M, N, 64, None, None, L.MOE_FP32, 0)
        assert L.moe_fp8_matmul_workspace_bytes(M, N, 64, L.MOE_BF16) == 0
    assert L.moe_fp8_matmul_workspace_bytes(2, 2, 40, L.MOE_BF16) == 0
    assert L.moe_fp8_matmul_workspace_bytes(2, 2, 64, L.MOE_FP32) == 0


def test_expert_refusals():
    T, H, I, E, k = 4, 64, 32, 8, 2
    need = L.moe_fp8_expert_ffn_workspace_bytes(T, H, I, E, k, 0)

    def f(x=FAKE, T=T, H=H, I=I, E=E, idx=FAKE, k=k, table=FAKE, shared=None, mask=None, y=FAKE, ws=FAKE, n=1 << 40):
        one = status(L.moe_fp8_expert_ffn, x, T, H, I, E, idx, k, table, shared, mask, y, ws, n)
        two = status(L.moe_fp8_expert_ffn_combine, x, T, H, I, E, idx, FAKE, k, table, shared, y, ws, n)
        assert one == two
        return one
    assert f(T=-1) == L.MOE_E_ARG
    for bad in (0, -32, 48, 16416):
        assert f(H=bad) == L.MOE_E_SHAPE and f(I=bad) == L.MOE_E_SHAPE
    assert f(E=0) == L.MOE_E_SHAPE and f(E=1025) == L.MOE_E_SHAPE and f(k=0) == L.MOE_E_SHAPE and f(k=9) == L.MOE_E_SHAPE
    assert f(T=16385, k=1) == L.MOE_E_SHAPE
    for name in ("x", "idx", "table", "y", "ws"):
        assert f(**{name: None}) == L.MOE_E_ARG
    for name in ("x", "shared", "y", "ws"):
        assert f(**{name: FAKE + 8}) == L.MOE_E_ARG
    assert f(n=need - 1) == L.MOE_E_NOMEM
    assert status(L.moe_fp8_expert_ffn_combine, FAKE, T, H, I, E, FAKE, None, k, FAKE, None, FAKE, FAKE, 1 << 40) == \
        L.MOE_E_ARG
    L.moe_fp8_expert_ffn(None, 0, H, I, E, None, k, None, None, None, None, None, 0)  # no tokens: nothing to do
    L.moe_fp8_expert_ffn_combine(None, 0, H, I, E, None, None, k, None, None, None, None, 0)
    assert L.moe_expert_bytes_fp8(256, 128) == 3 * 256 * 128 + 4 * 6 + 8
    assert L.moe_expert_bytes_fp8(160, 96) == 3 * 160 * 96 + 4 * 6 + 8
    for bad in ((0, 32), (48, 32), (32, 40)):
        assert L.moe_expert_bytes_fp8(*bad) == 0


# ------------------------------------------------------------------ the numpy forms
def test_values_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8kit.VALUES, ref, equal_nan=True)


def test_nearest_by_hand():
    u = np.array([0.0, 2.0 ** -10, 3 * 2.0 ** -10, 1.0, 1.0625, 1.0624, 1.1875, 448.0, 464.0, 1e9, 2.0 ** -11])
    assert GRID_at(u) == [0.0, 0.0, 2.0 ** -8, 1.0, 1.0, 1.0, 1.25, 448.0, 448.0, 448.0, 0.0]


def GRID_at(u):
    return fp8kit.GRID[fp8kit.nearest(u)].tolist()


def test_scales_by_hand():
    top = np.array([[0.0, 448.0, 449.0, 1.75, 1.76, 2.0 ** -149, np.inf, np.nan]])
    a = fp8kit.scale_of(top, "amax")[0]
    assert a[0] == 1 and a[1] == 1 and a[2] == np.float32(449 / 448) and a[5] == np.float32(2.0 ** -126)
    assert np.isnan(a[6]) and np.isnan(a[7])
    p = fp8kit.scale_of(top, "pow2")[0]
    assert p[:6].tolist() == [1, 1, 2, 2.0 ** -8, 2.0 ** -7, 2.0 ** -126]


def test_route_by_hand():
    l = np.array([[0.0, 3.0, 1.0, 1.0, 2.0, -1.0]], np.float32)
    idx, w = fp8kit.route(l, None, 3, "softmax", 1, 1, "max", True, 1.0)
    assert idx.tolist() == [[1, 4, 2]] and abs(w.sum() - 1) < 1e-12
    # groups (0,1), (2,3), (4,5): worth 3, 1, 2 by the largest; by the two largest sigmoids 1.45, 1.46, 1.15
    assert fp8kit.route(l, None, 2, "sigmoid", 3, 1, "max", False, 1.0)[0].tolist() == [[1, 0]]
    assert fp8kit.route(l, None, 2, "sigmoid", 3, 1, "top2", False, 1.0)[0].tolist() == [[2, 3]]
    b = np.array([0, -10, 0, 0, 0, 0.0])
    idx, w = fp8kit.route(l, b, 2, "sigmoid", 1, 1, "max", False, 2.0)
    assert idx.tolist() == [[4, 2]] and abs(w[0, 0] - 2 / (1 + np.exp(-2))) < 1e-12
