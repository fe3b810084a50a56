"""The runtime's FP8 layers without a GPU: what they refuse."""
import ctypes

import pytest
import torch

import synth
from routed_expert_streaming_amd import _lib as L
from routed_expert_streaming_amd.runtime import Fp8Linear, Fp8MoELayer, MoEStack, pack_fp8_expert, quantise_fp8

ROUTING = L.moe_routing(L.MOE_SCORE_SIGMOID, 1, 1, L.MOE_GROUP_MAX, 1, 1.0)


def test_quantise_refusals():
    w = torch.zeros((64, 96), dtype=torch.bfloat16)
    for bad in (w, w[0], w.double(), w.t()):  # not on the GPU, not a matrix, a type, columns apart
        with pytest.raises(ValueError):
            quantise_fp8(bad)


def test_pack_refusals():
    w, down = torch.zeros((64, 96), dtype=torch.bfloat16), torch.zeros((96, 64), dtype=torch.bfloat16)
    for args in ((w, w, w), (w, w[:32], down), (w, w, down)):  # shapes; and nothing here is on a GPU
        with pytest.raises(ValueError):
            pack_fp8_expert(*args)
    with pytest.raises(ValueError):
        pack_fp8_expert(w, w, down, slab=torch.zeros(16, dtype=torch.uint8))


def test_linear_refusals():
    w = torch.zeros((64, 96), dtype=torch.bfloat16)
    codes, scales = torch.zeros((64, 96), dtype=torch.uint8), torch.zeros((1, 1))
    for weight in (w, (codes, scales), (codes, scales.double()), (codes[:, :90], scales), (codes, torch.zeros((2, 1)))):
        with pytest.raises(ValueError):
            Fp8Linear(weight)
    with pytest.raises(ValueError):
        Fp8Linear(w, out_dtype=torch.float16)


def test_layer_refusals():
    router = torch.zeros((2, 96))
    w, down = torch.zeros((64, 96), dtype=torch.bfloat16), torch.zeros((96, 64), dtype=torch.bfloat16)
    for experts in ([(w, w, down)], [(w, w, down), (w[:32], w[:32], down)], [(w, w, down)] * 2):
        with pytest.raises(ValueError):
            Fp8MoELayer(router, experts, 1, ROUTING)
    with pytest.raises(ValueError):
        Fp8MoELayer(router, [(w, w, down)] * 2, 1, ROUTING, balance=torch.zeros(3))


def test_a_balance_needs_a_routing():
    with pytest.raises(ValueError):
        MoEStack(synth.get("tiny"), balance=torch.zeros((1, 16)))


def test_cache_formats():
    """A cache of FP8 slabs passes the checks of its description (the next one, of the host slabs, refuses this call);
    numbers between the formats do not."""
    ptrs = (ctypes.c_void_p * 4)()
    for fmt, want in ((L.MOE_FP8, "expert"), (3, "format"), (5, "format"), (-1, "format")):
        with pytest.raises(L.MoEError) as ei:
            L.moe_cache_create(L.moe_cache_desc(1, 4, 96, 64, 2, fmt), ctypes.addressof(ptrs), 0x1000, 0x1000, 0)
        assert ("format" in str(ei.value)) == (want == "format"), str(ei.value)
