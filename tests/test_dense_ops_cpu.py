"""The dense MXFP4 operators without a GPU: their refusals, and the numpy forms the GPU tests compare with."""
import numpy as np
import pytest
import torch

import oracle
from routed_expert_streaming_amd import _lib as L
from routed_expert_streaming_amd.runtime import MxLinear, pack_mx_expert, quantise_mx
from tests import mxkit

FAKE = 0x1000  # never dereferenced: the calls below fail validation or have nothing to do
ODD = FAKE + 2


def status(fn, *args):
    with pytest.raises(L.MoEError) as ei:
        fn(*args)
    return ei.value.status


def test_row_bytes():
    for K in (32, 64, 96, 128, 480, 512, 4096, 6144):
        assert L.moe_mx_row_bytes(K) == mxkit.row_bytes(K)
    for K in (0, -32, 33, 16):
        assert L.moe_mx_row_bytes(K) == 0
    H, I = 256, 128
    assert L.moe_expert_bytes_mx(H, I) == 2 * I * L.moe_mx_row_bytes(H) + H * L.moe_mx_row_bytes(I)


def test_quant_refusals():
    def q(x=FAKE, t=L.MOE_BF16, xs=128, rows=2, K=64, rule=0, out=FAKE, os=48, values=None):
        return status(L.moe_mx_quant, x, t, xs, rows, K, rule, out, os, values)
    assert q(rows=-1) == L.MOE_E_ARG
    assert q(t=L.MOE_MXFP4) == L.MOE_E_ARG and q(t=-1) == L.MOE_E_ARG
    assert q(rule=2) == L.MOE_E_ARG and q(rule=-1) == L.MOE_E_ARG
    for K in (0, -32, 48):
        assert q(K=K) == L.MOE_E_SHAPE
    assert q(x=None) == L.MOE_E_ARG and q(out=None) == L.MOE_E_ARG
    assert q(xs=112) == L.MOE_E_SHAPE and q(os=32) == L.MOE_E_SHAPE and q(xs=-128) == L.MOE_E_SHAPE
    assert q(t=L.MOE_FP32) == L.MOE_E_SHAPE  # 128 bytes hold half a row
    assert q(x=ODD) == L.MOE_E_ARG and q(out=ODD) == L.MOE_E_ARG and q(values=ODD) == L.MOE_E_ARG
    assert q(xs=136) == L.MOE_E_ARG and q(os=56) == L.MOE_E_ARG
    L.moe_mx_quant(None, L.MOE_BF16, 0, 0, 64, 0, None, 0)  # no rows: nothing to do


def test_matmul_refusals():
    def m(a=FAKE, at=L.MOE_BF16, as_=128, w=FAKE, ws=48, M=2, N=2, K=64, bias=None, y=FAKE, yt=L.MOE_FP32, ys=8):
        return status(L.moe_mx_matmul, a, at, as_, w, ws, M, N, K, bias, y, yt, ys, None, 0)
    assert m(M=-1) == L.MOE_E_ARG and m(N=-1) == L.MOE_E_ARG
    assert m(at=L.MOE_FP32) == L.MOE_E_ARG and m(yt=L.MOE_FP16) == L.MOE_E_ARG and m(yt=L.MOE_MXFP4) == L.MOE_E_ARG
    for K in (0, -64, 40):
        assert m(K=K) == L.MOE_E_SHAPE
    assert m(a=None) == L.MOE_E_ARG and m(w=None) == L.MOE_E_ARG and m(y=None) == L.MOE_E_ARG
    assert m(as_=112) == L.MOE_E_SHAPE and m(ws=32) == L.MOE_E_SHAPE and m(ys=4) == L.MOE_E_SHAPE
    assert m(at=L.MOE_MXFP4, as_=32) == L.MOE_E_SHAPE
    assert m(a=ODD) == L.MOE_E_ARG and m(w=ODD) == L.MOE_E_ARG and m(as_=136) == L.MOE_E_ARG and m(ws=56) == L.MOE_E_ARG
    assert m(y=ODD) == L.MOE_E_ARG and m(ys=10) == L.MOE_E_ARG and m(bias=ODD) == L.MOE_E_ARG
    assert m(M=(1 << 26) + 1) == L.MOE_E_SHAPE and m(N=(1 << 26) + 1, ys=1 << 40) == L.MOE_E_SHAPE
    assert m(K=(1 << 27) + 32) == L.MOE_E_SHAPE
    assert m(as_=(1 << 28) + 16) == L.MOE_E_SHAPE and m(ws=(1 << 28) + 16) == L.MOE_E_SHAPE
    for M, N in ((0, 2), (2, 0)):  # nothing to compute
        L.moe_mx_matmul(None, L.MOE_BF16, 0, None, 0, M, N, 64, None, None, L.MOE_FP32, 0)
        assert L.moe_mx_matmul_workspace_bytes(M, N, 64, L.MOE_BF16) == 0
    assert L.moe_mx_matmul_workspace_bytes(2, 2, 40, L.MOE_BF16) == 0


def test_block_norm_refusals():
    def n(add=FAKE, post=1, w_post=FAKE, gate=None, kind=0, resid=FAKE, out=FAKE, rt=L.MOE_FP32, w_pre=FAKE, T=2,
          H=64, eps=1e-6, x=FAKE, rows=None):
        return status(L.moe_block_norm, add, post, w_post, gate, kind, 1.0, resid, out, rt, w_pre, T, H, eps, x, rows)
    assert n(T=-1) == L.MOE_E_ARG and n(H=0) == L.MOE_E_ARG and n(H=(1 << 28) + 32) == L.MOE_E_SHAPE
    for eps in (-1.0, 2.0, float("nan")):
        assert n(eps=eps) == L.MOE_E_ARG
    assert n(rt=L.MOE_FP16) == L.MOE_E_ARG and n(kind=4) == L.MOE_E_ARG and n(kind=-1) == L.MOE_E_ARG
    assert n(post=0) == L.MOE_E_ARG  # w_post without a post norm
    assert n(resid=None) == L.MOE_E_ARG and n(out=None) == L.MOE_E_ARG
    assert n(add=None, x=None) == L.MOE_E_ARG  # nothing to write
    for kind in (L.MOE_GATE_CHANNEL, L.MOE_GATE_ROW, L.MOE_GATE_ELEMENT):
        assert n(kind=kind) == L.MOE_E_ARG
    assert n(kind=L.MOE_GATE_CHANNEL, gate=ODD) == L.MOE_E_ARG and n(kind=L.MOE_GATE_ELEMENT, gate=FAKE + 1) == L.MOE_E_ARG
    assert n(add=FAKE + 1) == L.MOE_E_ARG and n(resid=ODD) == L.MOE_E_ARG and n(w_pre=ODD) == L.MOE_E_ARG
    assert n(rows=FAKE, H=48) == L.MOE_E_SHAPE and n(rows=FAKE, add=ODD) == L.MOE_E_ARG
    assert n(rows=FAKE + 8) == L.MOE_E_ARG
    L.moe_block_norm(None, 0, None, None, 0, 1.0, None, None, L.MOE_FP32, None, 0, 64, 1e-6, None)  # no rows


def test_numpy_forms_agree_with_the_oracle():
    """pack/values against the oracle's own reading of an MXFP4 slab, quantise against its definition by hand."""
    rng = np.random.default_rng(5)
    H, I = 96, 64
    slab, parts = [], []
    for R, K in ((I, H), (I, H), (H, I)):
        c, s = mxkit.random_rows(rng, R, K, 0, 254)
        parts.append(mxkit.values(c, s))
        slab.append(mxkit.pack(c, s))
    flat = np.concatenate([np.stack([slab[0], slab[1]], 1).reshape(-1), slab[2].reshape(-1)])
    for which in range(3):
        assert np.array_equal(oracle.dequant(flat, H, I, which, 1), parts[which])
    x = np.zeros((1, 32))
    x[0, :9] = [4.0, 5.0, 5.001, 7.9, 0.25, 0.75, -0.25, -3.5, 0.2501]
    c, s = mxkit.quantise(x, "floor")
    assert s[0, 0] == 127 and c[0, :9].tolist() == [6, 6, 7, 7, 0, 2, 8, 14, 1]
    c, s = mxkit.quantise(x, "fit")  # halved: 2, 2.5, 2.5005, 3.95, .125, .375, .125, 1.75, .12505
    assert s[0, 0] == 128 and c[0, :9].tolist() == [4, 4, 5, 6, 0, 1, 8, 12, 0]


def test_runtime_refusals():
    w = torch.zeros((64, 96), dtype=torch.bfloat16)
    for bad in (w, w[0], w.double(), w.t()):  # not on the GPU, not a matrix, a type, columns apart
        with pytest.raises(ValueError):
            quantise_mx(bad)
    with pytest.raises(ValueError):
        MxLinear(w, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        MxLinear(w)
    down = torch.zeros((96, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pack_mx_expert(w, w, w)          # down has the wrong shape
    with pytest.raises(ValueError):
        pack_mx_expert(w, w[:32], down)
    with pytest.raises(ValueError):
        pack_mx_expert(w, w, down, slab=torch.zeros(16, dtype=torch.uint8))
    odd = torch.zeros((40, 96), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pack_mx_expert(odd, odd, odd.t())


@pytest.mark.parametrize("kind,M,N,K", [(L.MOE_MXFP4, 98, 1030, 20512), (L.MOE_BF16, 65, 130, 6176)])
def test_matmul_refuses_a_small_workspace(kind, M, N, K):
    """Sizes whose K is split: the parts' sums need a workspace, and less of it, none or one off its alignment is
    refused before anything runs."""
    a_stride = L.moe_mx_row_bytes(K) if kind == L.MOE_MXFP4 else 2 * K
    need = L.moe_mx_matmul_workspace_bytes(M, N, K, kind)
    assert need > 0 and need % (4 * M * N) == 0

    def m(ws, nbytes):
        return status(L.moe_mx_matmul, FAKE, kind, a_stride, FAKE, L.moe_mx_row_bytes(K), M, N, K, None, FAKE,
                      L.MOE_FP32, 4 * N, ws, nbytes)
    assert m(FAKE, need - 1) == L.MOE_E_NOMEM and m(FAKE, 0) == L.MOE_E_NOMEM and m(None, need) == L.MOE_E_NOMEM
    assert m(FAKE + 8, need) == L.MOE_E_ARG
