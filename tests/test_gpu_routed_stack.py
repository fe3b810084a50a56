"""Stacks of layers that route by scores, on the paths beside forward(): chained layers, with lookahead, with a CPU lane."""
import numpy as np
import pytest
import torch

import synth
from routed_expert_streaming_amd import _lib as L
from routed_expert_streaming_amd.runtime import MoEStack
from tests import fp8kit
from tests.test_gpu_chained import bits, lru_replay_chained, run_chain
from tests.test_gpu_fp8 import gpu  # noqa: F401
from tests.test_gpu_fp8_layers import f64
from tests.test_gpu_router_scored import weight_error

pytestmark = pytest.mark.gpu

LAYERS = 3


def how(cfg):
    """(a moe_routing, its balance [LAYERS, E], the arguments of fp8kit.route)"""
    g = torch.Generator().manual_seed(3)
    return (L.moe_routing(L.MOE_SCORE_SIGMOID, 8, 4, L.MOE_GROUP_TOP2, 1, 2.5),
            0.05 * torch.randn((LAYERS, cfg.experts), generator=g), ("sigmoid", 8, 4, "top2", True, 2.5))


def check_route(st, x, l, balance, rule):
    logits = fp8kit.logits(f64(x), f64(st.wr[l]), None if st.bias is None else f64(st.bias[l]))
    ri, rw = fp8kit.route(logits, balance[l].numpy(), st.k, *rule)
    assert np.array_equal(st.idx[l].cpu().numpy(), ri)
    assert (np.abs(f64(st.w[l]) - rw) <= weight_error(f64(x), f64(st.wr[l]), st.T, st.H) * rw).all()


def test_chained_with_lookahead():
    cfg = synth.get("decode1_stream")
    routing, balance, rule = how(cfg)
    whole = MoEStack(cfg, layers=LAYERS, cap=1.0, routing=routing, balance=balance)
    ref = run_chain(whole, 3, 0)
    xs = torch.from_numpy(ref[-1]["xs"].view(np.int16)).view(torch.bfloat16)
    for l in range(LAYERS):
        check_route(whole, xs[l], l, balance, rule)
    whole.close()
    streamed = MoEStack(cfg, layers=LAYERS, routing=routing, balance=balance)
    assert streamed.streaming
    try:
        for m in (0, 2, cfg.top_k):
            streamed.reset_cache()
            run = run_chain(streamed, 3, m)
            for a, b in zip(run, ref):
                assert (a["xs"] == b["xs"]).all() and (a["out"] == b["out"]).all() and (a["idx"] == b["idx"]).all()
            assert streamed.stats()[:2] == lru_replay_chained(run, LAYERS, streamed.C, m)
            if m:  # what is fetched ahead is the next layer's router on this layer's input
                xs = torch.from_numpy(run[-1]["xs"].view(np.int16)).view(torch.bfloat16)
                for l in range(LAYERS - 1):
                    logits = fp8kit.logits(f64(xs[l]), f64(streamed.wr[l + 1]),
                                           None if streamed.bias is None else f64(streamed.bias[l + 1]))
                    ahead = fp8kit.route(logits, balance[l + 1].numpy(), cfg.top_k, *rule)[0]
                    assert np.array_equal(run[-1]["pidx"][l + 1], ahead)
    finally:
        streamed.close()


@pytest.mark.parametrize("chained", [False, True])
def test_cpu_lane(chained):
    """Every other miss on the host: the choice is the definition's, the outputs those of the same routing with all
    experts on the GPU, to what the two lanes' sums differ by."""
    cfg = synth.get("decode1_stream")
    routing, balance, rule = how(cfg)
    st = MoEStack(cfg, layers=LAYERS, cpu_lane=4, routing=routing, balance=balance)
    whole = MoEStack(cfg, layers=LAYERS, cap=1.0, routing=routing, balance=balance)
    try:
        assert st.streaming and st.lane
        st.lane_pick = lambda l, misses: misses[::2]
        out, want = st.new_output(), whole.new_output()
        n = 0
        for s in range(2):
            x = st.make_inputs(s)
            if chained:
                resid, xs = st.chain_buffers()
                r = st.forward_chained(x[0], xs, resid, out)
                x = xs
            else:
                r = st.forward(x, out)
            torch.cuda.synchronize()
            n += r.cpu_experts
            for l in range(LAYERS):
                check_route(st, x[l], l, balance, rule)
                whole.idx[l].copy_(st.idx[l])
                whole.w[l].copy_(st.w[l])
                whole.ffn_combine(x, l, want)
            torch.cuda.synchronize()
            assert ((out.float() - want.float()).abs().amax((1, 2)) <= 2e-2 * want.float().abs().amax((1, 2))).all()
        assert n > 0
        st.lane_pick = lambda l, misses: []  # nothing on the host: the same bits
        if not chained:
            x = st.make_inputs(5)
            st.forward(x, out)
            whole.forward(x, want)
            torch.cuda.synchronize()
            assert (bits(out) == bits(want)).all()
    finally:
        st.close()
        whole.close()
