"""The dense MXFP4 operators through the runtime: the views, slabs and pools that its documentation allows."""
import numpy as np
import pytest
import torch

import oracle
import synth
from routed_expert_streaming_amd import _lib as L
from routed_expert_streaming_amd.runtime import RMS_EPS, BlockNorms, MoEStack, MxLinear, pack_mx_expert, quantise_mx
from tests import mxkit

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def shifted(t, elements=1):
    """t's values in a contiguous view that begins `elements` elements into its storage."""
    flat = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)
    flat[elements:] = t.flatten()
    return flat[elements:].view(t.shape)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantise_mx_takes_any_view(dtype):
    """Views that begin off a 16-byte boundary, whose rows lie an odd number of elements apart, or that repeat a row."""
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn((7, 96), generator=g, device="cuda").to(dtype)
    want = quantise_mx(w)
    wide = torch.zeros((7, 101), dtype=dtype, device="cuda")
    wide[:, 3:99] = w
    for view in (shifted(w), shifted(w, 3), wide[:, 3:99]):
        assert torch.equal(view, w)
        assert torch.equal(quantise_mx(view), want)
        assert torch.equal(MxLinear(view).rows, want)
    assert torch.equal(quantise_mx(shifted(w[:1])), want[:1])
    assert torch.equal(quantise_mx(w[2:3].expand(5, 96)), want[2:3].expand(5, -1))


@pytest.mark.parametrize("quantise_input", [False, True])
def test_mx_linear_takes_any_view(quantise_input):
    g = torch.Generator(device="cuda").manual_seed(4)
    N, K = 65, 160
    lin = MxLinear(torch.randn((N, K), generator=g, device="cuda"), quantise_input=quantise_input,
                   out_dtype=torch.float32)
    for shape in ((K,), (1, K), (5, K), (2, 3, K)):
        x = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        for n in (1, 3):
            assert torch.equal(lin(shifted(x, n)), lin(x))
    x = torch.randn((4, K), generator=g, device="cuda").to(torch.bfloat16)
    assert torch.equal(lin(x[1:2].expand(3, K)), lin(x[1:2]).expand(3, N))
    rows = quantise_mx(x)
    assert torch.equal(lin(shifted(rows, 8)), lin(rows))


def test_pack_mx_expert_refused_leaves_the_slab():
    """A slot of a live pool: matrices that are refused (the last one a transposed view, a wrong type, on the host) must
    not leave half an expert behind."""
    g = torch.Generator(device="cuda").manual_seed(5)
    H, I = 96, 64
    w1, w3, w2 = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((I, H), (I, H), (H, I)))
    slab = torch.full((L.moe_expert_bytes_mx(H, I),), 0xA5, dtype=torch.uint8, device="cuda")
    for bad in ((w1, w3, w2.t().contiguous().t()), (w1, w3.double(), w2), (w1, w3, w2.cpu()), (w1, w3.cpu(), w2)):
        with pytest.raises(ValueError):
            pack_mx_expert(*bad, slab=slab)
        assert (slab == 0xA5).all()
    with pytest.raises(L.MoEError):
        pack_mx_expert(w1, w3, w2, slab=slab, scale_rule=2)
    assert (slab == 0xA5).all()
    wide = torch.full((slab.numel() + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    with pytest.raises(L.MoEError):
        pack_mx_expert(w1, w3, w2, slab=wide[8:8 + slab.numel()])  # off a 16-byte boundary
    assert (wide == 0xA5).all()
    pack_mx_expert(w1, w3, w2, slab=slab)
    assert torch.equal(slab, pack_mx_expert(shifted(w1), shifted(w3), shifted(w2)))


@pytest.fixture
def stacks():
    """A streamed and a resident stack of one configuration, closed after a failure has been shown: the views of the
    host pool die with them."""
    cfg = synth.get("tiny", fmt=1, layers=2, cap=0.5)
    both = MoEStack(cfg), MoEStack(cfg, cap=1.0)
    yield cfg, *both
    for st in both:
        st.close()


def test_a_streamed_stack_runs_a_users_experts(stacks):
    """Matrices of one's own packed into the pinned host pool of a streamed stack (and into the device pool of a
    resident one): the routed layers compute with them.  One expert has blocks of zeros."""
    cfg, streamed, resident = stacks
    assert streamed.streaming and not resident.streaming
    g = torch.Generator(device="cuda").manual_seed(6)
    H, I, E = streamed.H, streamed.I, streamed.E
    for l in range(2):
        for e in range(E):
            mats = [(torch.randn(s, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
                    for s in ((I, H), (I, H), (H, I))]
            if e == 3:
                mats[0][5, :64] = 0.0
                mats[2][:, 32:64] = 0.0
            to = torch.from_numpy(streamed.host_pool_slabs(l)[e])
            assert pack_mx_expert(*mats, slab=to).data_ptr() == to.data_ptr()
            pack_mx_expert(*mats, slab=resident.pool[l * E + e])
            assert torch.equal(resident.pool[l * E + e].cpu(), to)
    x, out, out2 = streamed.make_inputs(0), streamed.new_output(), streamed.new_output()
    streamed.forward(x, out)
    resident.forward(x, out2)
    torch.cuda.synchronize()
    for l in range(2):
        bits = x[l].view(torch.int16).cpu().numpy().view(np.uint16)
        ref = oracle.moe_layer(bits, streamed.wr[l].cpu().numpy(), None, cfg.top_k,
                               [np.array(s) for s in streamed.host_pool_slabs(l)], None, I, fmt=1)
        assert (streamed.idx[l].cpu().numpy() == ref["idx"]).all()
        for o in (out, out2):
            err = np.abs(o[l].double().cpu().numpy() - ref["out64"]).max()
            assert err <= 2e-2 * np.abs(ref["out64"]).max()
    refused = torch.from_numpy(np.full(streamed.slab, 0xA5, np.uint8))
    for bad in (refused[:-1], refused.view(torch.int8)):
        with pytest.raises(ValueError):
            pack_mx_expert(*mats, slab=bad)
    assert (refused == 0xA5).all()


def learned(st, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [1 + 0.2 * torch.randn((st.L, st.H), generator=g, device="cuda") for _ in range(2)]
    return BlockNorms(*w, torch.rand((st.L, st.H), generator=g, device="cuda"), 0.5)


def chain(st, h0, norms, lookahead=0):
    resid, xs = st.chain_buffers()
    out = st.new_output()
    st.forward_chained(h0, xs, resid, out, lookahead, norms=norms)
    torch.cuda.synchronize()
    return resid, xs, out


def test_chained_norms_need_their_input_norm(stacks):
    _, streamed, _ = stacks
    resid, xs = streamed.chain_buffers()
    resid.fill_(7.0)
    with pytest.raises(ValueError):
        streamed.forward_chained(streamed.make_inputs(0)[0], xs, resid, streamed.new_output(), norms=BlockNorms(None))
    assert (resid == 7.0).all()


def test_chained_norms_after_the_last_layer(stacks):
    """The stream does not hold the last layer's output; the call that the documentation gives for it does the rest."""
    _, streamed, st = stacks
    h0, norms = st.make_inputs(0)[0], learned(st, 8)
    resid, xs, out = chain(st, h0, norms)
    for t in (norms.post, norms.gate):
        t[-1] = float("nan")  # not read by the step
    again = chain(st, h0, norms)
    for a, b in zip((resid, xs, out), again):
        assert torch.equal(a, b)
    last = learned(st, 9)
    x = torch.empty((st.T, st.H), dtype=torch.bfloat16, device="cuda")
    before = resid.double().cpu().numpy()
    L.moe_block_norm(out[-1], 1, last.post[-1], last.gate[-1], L.MOE_GATE_CHANNEL, 0.5, resid, resid, L.MOE_FP32,
                     last.pre[-1], st.T, st.H, RMS_EPS, x, None, torch.cuda.current_stream())
    host = [t.double().cpu().numpy() for t in (out[-1], last.post[-1], last.gate[-1], last.pre[-1], resid, x)]
    want = mxkit.block_norm(host[0], True, host[1], host[2], 0.5, before, RMS_EPS)
    # 8 squares a thread, 6 sums of a wave, mean, eps, root, reciprocal and three products: 21 roundings
    u = 24 * 2.0 ** -24
    assert (np.abs(host[4] - want) <= u * np.abs(want - before) + 2.0 ** -24 * np.abs(want)).all()
    final = mxkit.norm(host[4], host[3], RMS_EPS)
    assert (np.abs(host[5] - final) <= (2.0 ** -8 * (1 + u) + u) * np.abs(final)).all()


@pytest.mark.parametrize("lookahead", [0, 1])
def test_chained_norms_streamed_equal_resident(lookahead):
    cfg = synth.get("tiny", fmt=1, layers=3, cap=0.75)
    streamed, resident = MoEStack(cfg), MoEStack(cfg, cap=1.0)
    try:
        assert streamed.streaming and not resident.streaming
        for step in range(2):
            h0, norms = resident.make_inputs(step)[0], learned(resident, 10 + step)
            for a, b in zip(chain(streamed, h0, norms, lookahead), chain(resident, h0, norms)):
                assert torch.equal(a, b)
    finally:
        streamed.close()
        resident.close()
