"""The FP8 operators as layers and together: each against its definition in 64 bits, and as parts of the framework's own
paths (a cached pool, a stack of layers, a captured graph)."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from routed_expert_streaming_amd import _lib as L
from routed_expert_streaming_amd.runtime import (RMS_EPS, Fp8Linear, Fp8MoELayer, MoEStack, PinnedHost, pack_fp8_expert,
                                                 quantise_fp8)
from tests import fp8kit
from tests.test_gpu_fp8 import dev, gpu, hidden, routing  # noqa: F401
from tests.test_gpu_router_scored import weight_error

pytestmark = pytest.mark.gpu


def matrix(seed, rows, K, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, K), generator=g) * (1.5 / K ** 0.5)).to(dtype).cuda()


def f64(t):
    return t.double().cpu().numpy()


def check_linear(x, y, codes, scales, bias):
    """y = x W^T + bias within the sums' error and y's rounding; x bf16."""
    K = x.shape[-1]
    va = fp8kit.values(*fp8kit.quantise(f64(x)), 1)
    vw = fp8kit.values(codes.cpu().numpy(), scales.cpu().numpy(), 128)
    want, mag = va @ vw.T, np.abs(va) @ np.abs(vw).T
    if bias is not None:
        want, mag = want + f64(bias), mag + np.abs(f64(bias))
    bf16 = y.dtype == torch.bfloat16
    off = (fp8kit.sum_error(K) + fp8kit.cores_error(bf16) + 2.0 ** -24) * mag
    assert (np.abs(f64(y) - want) <= off + (2.0 ** -8 if bf16 else 2.0 ** -24) * (np.abs(want) + off)).all()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_linear(out):
    N, K = 200, 272
    w, bias = matrix(1, N, K), torch.linspace(-1, 1, N).cuda()
    lin = Fp8Linear(w, bias, out_dtype=out)
    for shape in ((1,), (2, 3), (40,), (0,)):
        x = hidden(len(shape), int(np.prod(shape)), K).cuda()
        y = lin(x.reshape(*shape, K))
        assert y.shape == (*shape, N) and y.dtype == out
        check_linear(x, y.reshape(-1, N), lin.codes, lin.scales, bias)
        # given as codes the rows may meet another kernel, which adds in another order: the same bound, not the same bits
        a = quantise_fp8(x, 1)
        coded = lin(a)
        check_linear(x, coded, lin.codes, lin.scales, bias)
        packed = (a[0], a[1].contiguous())  # scale rows the product does not take as they lie
        assert torch.equal(lin(packed), coded)
    wide = hidden(9, 7, K + 8).cuda()
    for view in (wide[:, :K], wide[:, 3:K + 3], wide[::2, :K]):  # strided, off its alignment
        assert torch.equal(lin(view), lin(view.contiguous().clone()))
    again = Fp8Linear((lin.codes.view(torch.float8_e4m3fn), lin.scales), bias, out_dtype=out)
    assert torch.equal(again(wide[:, :K]), lin(wide[:, :K]))
    for bad in (wide, wide[:, :K].float(), wide[:, :K].cpu(), (lin.codes[:3, :128], lin.scales[:1]),
                (a[0].view(torch.int8), a[1])):
        with pytest.raises(ValueError):
            lin(bad)
    for other in (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int8):  # bytes of another meaning
        with pytest.raises(ValueError):
            Fp8Linear((lin.codes.view(other), lin.scales))


def test_pack_places_every_block():
    H, I = 288, 160
    w = [matrix(i, *s) for i, s in enumerate(((I, H), (I, H), (H, I)))]
    for rule, name in ((L.MOE_FP8_SCALE_AMAX, "amax"), (L.MOE_FP8_SCALE_POW2, "pow2")):
        want = fp8kit.slab([fp8kit.quantise(f64(m), 128, name) for m in w])
        got = pack_fp8_expert(*w, scale_rule=rule)
        assert np.array_equal(got.cpu().numpy(), want)
        host = torch.empty(len(want), dtype=torch.uint8)
        assert pack_fp8_expert(*w, slab=host, scale_rule=rule) is not None
        assert np.array_equal(host.numpy(), want)
    strided = torch.zeros((I, H + 24), dtype=torch.bfloat16, device="cuda")
    strided[:, 8:H + 8] = w[0]
    assert torch.equal(pack_fp8_expert(strided[:, 8:H + 8], w[1], w[2]), pack_fp8_expert(*w))


class Layer:
    """A layer, the numbers its slabs hold and its routing rule."""

    def __init__(self, H, I, E, k, shared, groups, top):
        self.E, self.H, self.I, self.k, self.groups, self.top = E, H, I, k, groups, top
        triples = [[matrix(100 * e + i, *s) for i, s in enumerate(((I, H), (I, H), (H, I)))] for e in range(E + shared)]
        self.parts = [[fp8kit.quantise(f64(m), 128) for m in t] for t in triples]
        self.router = matrix(7, E, H, torch.float32)
        self.balance = torch.linspace(-0.02, 0.02, E).cuda()[torch.randperm(E, generator=torch.Generator().manual_seed(1))]
        how = L.moe_routing(L.MOE_SCORE_SIGMOID, groups, top, L.MOE_GROUP_TOP2, 1, 2.5)
        self.layer = Fp8MoELayer(self.router, triples[:E], k, how, balance=self.balance,
                                 shared=triples[E] if shared else None)
        self.shared = shared

    def check_route(self, x, idx, w):
        l = fp8kit.logits(f64(x), f64(self.router), None)
        ri, rw = fp8kit.route(l, self.balance.cpu().numpy(), self.k, "sigmoid", self.groups, self.top, "top2", True, 2.5)
        assert np.array_equal(idx.cpu().numpy(), ri)
        error = weight_error(f64(x), f64(self.router), x.shape[0], self.H)
        assert (np.abs(f64(w) - rw) <= error * rw).all()

    def check(self, x, idx, w, out):
        """out against the experts' feed-forward of the given routing."""
        idx, w = idx.cpu().numpy(), f64(w)
        T = len(idx)
        xq = fp8kit.values(*fp8kit.quantise(f64(x)), 1)
        want, off, mag = np.zeros((T, self.H)), np.zeros((T, self.H)), np.zeros((T, self.H))
        for e in range(self.E + self.shared):
            t, i = np.nonzero(idx == e) if e < self.E else (np.arange(T), None)
            if len(t):
                y, err = fp8kit.feed_forward(xq[t], self.parts[e])
                by = w[t, i][:, None] if e < self.E else 1.0
                want[t] += by * y
                off[t] += by * err
                mag[t] += by * (np.abs(y) + err)
        off += (self.k + 2) * 2.0 ** -24 * mag
        assert (np.abs(f64(out) - want) <= off + 2.0 ** -8 * (np.abs(want) + off)).all()


@pytest.fixture(scope="module")
def layer():
    return Layer(384, 160, 24, 4, True, 4, 2)


@pytest.mark.parametrize("T", [0, 1, 3, 24, 210, 700])
def test_layer(layer, T):
    x = hidden(T, T, layer.H).cuda()
    out = layer.layer(x)
    assert out.shape == x.shape
    if T:
        idx, w = layer.layer.route(x)
        layer.check_route(x, idx, w)
        layer.check(x, idx, w, out)
    for bad in (x.float(), x[:, :128], x.cpu()):
        with pytest.raises(ValueError):
            layer.layer(bad)


@pytest.mark.parametrize("T", [1, 24, 210])
def test_the_operators_together(layer, T):
    """A block as a model runs it: a projection, the norm with the residual stream, the routed experts, the next norm and
    the logits; every step against its definition on the step's own inputs, then as a captured graph, replayed with eager
    steps between."""
    H = layer.H
    proj, head = Fp8Linear(matrix(51, H, H)), Fp8Linear(matrix(52, 504, H), out_dtype=torch.float32)
    x0 = [hidden(60 + i, T, H).cuda() for i in range(2)]
    x, resid = x0[0].clone(), torch.zeros((T, H), device="cuda")
    ones = torch.ones(H, device="cuda")

    def norm(add, xn):
        L.moe_block_norm(add, 0, None, None, L.MOE_GATE_NONE, 1.0, resid, resid, L.MOE_FP32, ones, T, H, RMS_EPS, xn,
                         None, torch.cuda.current_stream())
        return xn

    def step():
        resid.copy_(x.float())
        a = proj(x)
        n1 = norm(a, torch.empty_like(x))
        m = layer.layer(n1)
        n2 = norm(m, torch.empty_like(x))
        return a, n1, m, n2, head(n2)
    a, n1, m, n2, y = step()
    check_linear(x, a, proj.codes, proj.scales, None)
    idx, w = layer.layer.route(n1)
    layer.check_route(n1, idx, w)
    layer.check(n1, idx, w, m)
    check_linear(n2, y, head.codes, head.scales, None)
    want = []
    for v in x0:
        x.copy_(v)
        want.append(step()[-1].clone())
    assert torch.equal(want[0], y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()[-1]
    for i in (0, 1, 0, 1, 1):
        x.copy_(x0[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, want[i])
        assert torch.equal(step()[-1], want[i])
        torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 9, 150])
def test_streamed_experts(T):
    """FP8 slabs through the expert cache, with fewer slots than experts, in waves; the same bits as all at once."""
    H, I, E, C, k = 256, 96, 10, 4, 3
    triples = [[matrix(10 * e + i, *s) for i, s in enumerate(((I, H), (I, H), (H, I)))] for e in range(E)]
    n = L.moe_expert_bytes_fp8(H, I)
    host = PinnedHost(E * n)
    whole = torch.empty((E, n), dtype=torch.uint8, device="cuda")
    for e, t in enumerate(triples):
        pack_fp8_expert(*t, slab=torch.from_numpy(host.array[e * n:(e + 1) * n]))
        pack_fp8_expert(*t, slab=whole[e])
    x, idx = hidden(T, T, H).cuda(), dev(routing(np.random.default_rng(T), T, E, k))
    need = L.moe_fp8_expert_ffn_workspace_bytes(T, H, I, E, k, 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream()
    table = dev(whole.data_ptr() + n * np.arange(E))
    want = torch.zeros((T * k, H), device="cuda")
    L.moe_fp8_expert_ffn(x, T, H, I, E, idx, k, table, None, None, want, ws, need, s)

    ptrs = (ctypes.c_void_p * E)(*(host.ptr + e * n for e in range(E)))
    pool = torch.empty((C, n), dtype=torch.uint8, device="cuda")
    slots = torch.zeros((1, E), dtype=torch.int64, device="cuda")
    copies = torch.cuda.Stream()
    cache = L.moe_cache_create(L.moe_cache_desc(1, E, H, I, C, L.MOE_FP8), ctypes.addressof(ptrs), pool, slots, copies)
    try:
        needed = sorted(set(idx.flatten().tolist()))
        for _ in range(2):
            y = torch.full((T * k, H), 3.0, device="cuda")
            for wave in (needed[i:i + C] for i in range(0, len(needed), C)):
                mask = np.zeros(E, np.uint8)
                mask[wave] = 1
                L.moe_cache_prefetch(cache, 0, wave, s)
                L.moe_fp8_expert_ffn(x, T, H, I, E, idx, k, slots, None, dev(mask), y, ws, need, s)
                L.moe_cache_release(cache, 0, s)
            torch.cuda.synchronize()
            assert torch.equal(y, want)
    finally:
        torch.cuda.synchronize()
        L.moe_cache_destroy(cache)
        host.free()


@pytest.mark.parametrize("cap", [1.0, 0.5])
def test_stack_routed_by_scores(cap):
    """A stack whose layers route by scores: the choice is the definition's, whether all experts are resident or half of
    them, and the outputs are those of the experts on it."""
    layers = 3
    cfg = synth.get("tiny", layers=layers)
    balance = torch.linspace(-0.1, 0.1, layers * 16).view(layers, 16)
    how = L.moe_routing(L.MOE_SCORE_SIGMOID, 4, 2, L.MOE_GROUP_MAX, 1, 1.5)
    st = MoEStack(cfg, layers=layers, cap=cap, routing=how, balance=balance)
    try:
        x = st.make_inputs(0)
        out = st.new_output()
        st.forward(x, out)
        torch.cuda.synchronize()
        for l in range(layers):
            ri, rw = fp8kit.route(fp8kit.logits(f64(x[l]), f64(st.wr[l]), None), balance[l].numpy(), st.k, "sigmoid", 4, 2,
                                  "max", True, 1.5)
            assert np.array_equal(st.idx[l].cpu().numpy(), ri)
            assert (np.abs(f64(st.w[l]) - rw) <= weight_error(f64(x[l]), f64(st.wr[l]), st.T, st.H) * rw).all()
        first = out.clone()
        idx, w = st.idx.clone(), st.w.clone()
        if cap == 1.0:
            for l in range(layers):
                st.idx[l].copy_(idx[l])
                st.w[l].copy_(w[l])
                st.ffn(x, l)
                st.combine(l, out)
            torch.cuda.synchronize()
            assert torch.equal(out, first)
        else:
            whole = MoEStack(cfg, layers=layers, cap=1.0, routing=how, balance=balance)
            whole.forward(x, out)
            torch.cuda.synchronize()
            assert torch.equal(whole.idx, idx) and torch.equal(out, first)
            whole.close()
    finally:
        st.close()
