"""Routing by scores on the GPU against its definition in 64 bits: experts equal, weights within weight_error() of it."""
import numpy as np
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from tests import fp8kit

pytestmark = pytest.mark.gpu



def weight_error(x, w, T, H):
    """How far a token's weights may be off, relative to themselves [T, 1]: the scale's product and the rounding to 32 bits
    (2^-24 each), and what the 64-bit exponentials differ by; of more than a few tokens four times its logits' error (a
    softmax or a renormalised weight moves by at most twice it, to first order, and the bound is below 2^-4).

    That error, where the logits are summed on the bf16 matrix cores: per 64 columns two sums of 32 products, each off by at
    most 6 * 2^-23 of its terms' magnitudes (and four more of 2^-7 of it), one addition per 64 columns to the total (2^-24),
    and one rounding of the logit; the sum of magnitudes is at most |x| |w|."""
    if T <= FEW:
        return 2.0 ** -23
    big = np.sqrt((x ** 2).sum(1, keepdims=True)) * np.sqrt((w ** 2).sum(1).max())
    logit = (16 + (H / 64 + 1) / 2) * 2.0 ** -23 * big + 2.0 ** -23 * np.abs(x @ w.T).max(1, keepdims=True)
    assert logit.max() < 2.0 ** -4
    return 2.0 ** -23 + 4 * logit


FEW = 8  # tokens up to which every logit is summed in 64 bits
SCORE = {"softmax": L.MOE_SCORE_SOFTMAX, "sigmoid": L.MOE_SCORE_SIGMOID}
RULE = {"max": L.MOE_GROUP_MAX, "top2": L.MOE_GROUP_TOP2}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


class Call:
    """One call's device buffers; run() enqueues it on a stream."""

    def __init__(self, x, w, bias, balance, k, score, groups, top, rule, renorm, scale):
        self.layers, self.T, self.H = x.shape
        self.E, self.k = w.shape[1], k
        self.x, self.w = dev(x, torch.bfloat16), dev(w, torch.float32)
        self.bias = None if bias is None else dev(bias, torch.float32)
        self.balance = None if balance is None else dev(balance, torch.float32)
        self.how = L.moe_routing(SCORE[score], groups, top, RULE[rule], int(renorm), scale)
        self.idx = torch.full((self.layers * self.T + 1, k), -7, dtype=torch.int32, device="cuda")
        self.wt = torch.full((self.layers * self.T + 1, k), 7.0, device="cuda")
        self.need = L.moe_router_scored_workspace_bytes(self.layers, self.T, self.E, self.H)
        self.ws = torch.full((self.need + 64,), 0xA5, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        L.moe_router_scored(self.x, self.layers, self.T, self.H, self.w, self.bias, self.balance, self.E, self.k,
                            self.how, self.idx, self.wt, self.ws, self.need,
                            torch.cuda.current_stream() if stream is None else stream)
        return self

    def result(self):
        torch.cuda.synchronize()
        assert (self.idx[-1] == -7).all() and (self.wt[-1] == 7.0).all() and (self.ws[self.need:] == 0xA5).all()
        shape = (self.layers, self.T, self.k)
        return self.idx[:-1].cpu().numpy().reshape(shape), self.wt[:-1].double().cpu().numpy().reshape(shape)


def inputs(seed, layers, T, H, E, balance=True, bias=False, spread=1.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((layers, T, H))).to(torch.bfloat16).double().numpy()
    w = (rng.standard_normal((layers, E, H)) * (spread / H ** 0.5)).astype(np.float32).astype(np.float64)
    b = (rng.standard_normal((layers, E))).astype(np.float32) if bias else None
    c = (0.1 * rng.standard_normal((layers, E))).astype(np.float32) if balance else None
    return x, w, b, c


def check(call, x, w, bias, balance, k, score, groups, top, rule, renorm, scale):
    idx, wt = call.run().result()
    for l in range(len(x)):
        lg = fp8kit.logits(x[l], w[l], None if bias is None else bias[l].astype(np.float64))
        ri, rw = fp8kit.route(lg, None if balance is None else balance[l], k, score, groups, top, rule, renorm, scale)
        assert np.array_equal(idx[l], ri)
        assert (np.abs(wt[l] - rw) <= weight_error(x[l], w[l], x.shape[1], x.shape[2]) * np.abs(rw) + 1e-45).all()


CASES = [  # layers, T, H, E, k, groups, top
    (1, 1, 32, 1, 1, 1, 1), (1, 1, 64, 8, 8, 1, 1), (1, 3, 96, 16, 2, 4, 1), (2, 5, 1056, 60, 6, 5, 2),
    (1, 1, 4096, 128, 8, 1, 1), (3, 32, 256, 64, 4, 64, 7), (1, 33, 256, 65, 5, 13, 3), (1, 32, 6144, 256, 8, 8, 4),
    (1, 47, 2080, 160, 6, 8, 3), (2, 70, 64, 256, 64, 2, 1), (1, 200, 512, 320, 10, 10, 4), (1, 300, 96, 512, 3, 32, 9),
    (1, 129, 160, 1000, 9, 4, 2), (1, 40, 64, 1024, 64, 64, 64), (1, 2, 16384, 24, 3, 6, 2), (5, 64, 128, 72, 8, 6, 6)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("layers,T,H,E,k,groups,top", CASES)
def test_route(layers, T, H, E, k, groups, top, score):
    for i, (rule, renorm, scale, balance, bias) in enumerate([("max", True, 1.0, True, False),
                                                              ("top2", False, 2.5, False, True)]):
        if rule == "top2" and E // groups < 2 and top < groups:
            rule = "max"
        x, w, b, c = inputs(1000 * T + E + i, layers, T, H, E, balance, bias)
        args = (k, score, groups, top, rule, renorm, scale)
        check(Call(x, w, b, c, *args), x, w, b, c, *args)


@pytest.mark.parametrize("T", [2, 70])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_index(score, T):
    """Experts with the same router rows, within a lane's and in different lanes, groups of equal worth, all-equal
    scores."""
    x, w, _, _ = inputs(5, 1, T, 128, 256, False)
    w[0, 64:128] = w[0, :64]
    w[0, 129] = w[0, 130] = w[0, 3]
    for args in ((12, score, 1, 1, "max", True, 1.0), (12, score, 4, 2, "max", True, 1.0),
                 (12, score, 4, 2, "top2", False, 1.0)):
        check(Call(x, w, None, None, *args), x, w, None, None, *args)
    w[:] = 0
    for args in ((9, score, 1, 1, "max", True, 1.0), (9, score, 8, 3, "top2", True, 4.0)):
        check(Call(x, w, None, None, *args), x, w, None, None, *args)


@pytest.mark.parametrize("T", [3, 50])
def test_saturated_scores(T):
    """Logits whose 32-bit scores would all be 1 or 0: 64 bits still tell them apart; where they do not either, the
    lower index wins, and a token whose scores are all zero gets zeros."""
    x, w, _, c = inputs(9, 1, T, 64, 40, True, spread=25.0)
    for balance in (None, c, 1e-7 * c):
        for args in ((7, "sigmoid", 1, 1, "max", True, 1.0), (7, "sigmoid", 5, 3, "top2", True, 1.0),
                     (7, "softmax", 5, 3, "max", False, 1.0)):
            check(Call(x, w, None, balance, *args), x, w, None, balance, *args)
    x[:], w[:] = 1.0, -32.0  # logits -2048: the sigmoids are zero
    call = Call(x, w, None, None, 3, "sigmoid", 1, 1, "max", True, 1.0)
    idx, wt = call.run().result()
    assert (idx == np.arange(3)).all() and (wt == 0).all()


@pytest.mark.parametrize("T", [2, 40])
def test_infinite_balance_and_nan(T):
    x, w, _, c = inputs(11, 1, T, 64, 48, True)
    c[0, 5:40] = -np.inf  # only 13 experts left
    args = (16, "sigmoid", 1, 1, "max", True, 1.0)
    check(Call(x, w, None, c, *args), x, w, None, c, *args)
    c[0, :24] = -np.inf   # the first two groups are worth nothing
    args = (6, "sigmoid", 4, 2, "top2", True, 1.0)
    check(Call(x, w, None, c, *args), x, w, None, c, *args)
    c[0, 7] = np.nan      # ranks first; nothing leaves its buffers
    idx, wt = Call(x, w, None, c, 6, "sigmoid", 4, 2, "top2", True, 1.0).run().result()
    assert (idx[0, :, 0] == 7).all() and ((idx >= 0) & (idx < 48)).all()


def test_layers_equal_single_calls():
    for T in (4, 80):
        x, w, b, c = inputs(21, 3, T, 256, 96, True, True)
        args = (6, "sigmoid", 6, 3, "top2", True, 2.5)
        idx, wt = Call(x, w, b, c, *args).run().result()
        for l in range(3):
            i1, w1 = Call(x[l:l + 1], w[l:l + 1], b[l:l + 1], c[l:l + 1], *args).run().result()
            assert np.array_equal(idx[l], i1[0]) and np.array_equal(wt[l], w1[0])


def test_same_experts_as_the_other_router():
    """Softmax scores without groups choose as moe_router_topk does."""
    for T in (3, 100):
        x, w, b, _ = inputs(31, 1, T, 512, 64, False, True)
        call = Call(x, w, b, None, 6, "softmax", 1, 1, "max", True, 1.0)
        idx, wt = call.run().result()
        i2 = torch.empty((T, 6), dtype=torch.int32, device="cuda")
        w2 = torch.empty((T, 6), device="cuda")
        need = L.moe_router_workspace_bytes(T, 64)
        L.moe_router_topk(call.x, T, 512, call.w, call.bias, 64, 6, i2, w2, torch.empty(need, dtype=torch.uint8,
                          device="cuda"), need, torch.cuda.current_stream())
        assert np.array_equal(idx[0], i2.cpu().numpy())
        assert np.abs(wt[0] - w2.double().cpu().numpy()).max() < 1e-6


def test_streams_and_graphs():
    """Two calls at once on streams of their own, and a captured one replayed between eager calls, equal the eager
    results."""
    for T in (1, 32, 150):
        calls, want = [], []
        for i in range(2):
            x, w, b, c = inputs(41 + i, 2, T, 320, 128, True, True)
            call = Call(x, w, b, c, 8, "sigmoid", 8, 3, "top2", True, 1.5)
            want.append([a.copy() for a in call.run().result()])
            calls.append(call)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(3):
            for call, s in zip(calls, streams):
                call.idx[:-1].fill_(-1)
                torch.cuda.synchronize()
                call.run(s)
        for call, r in zip(calls, want):
            got = call.result()
            assert np.array_equal(got[0], r[0]) and np.array_equal(got[1], r[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for call in calls:
                call.run()
        for _ in range(3):
            for call in calls:
                call.idx[:-1].fill_(-1)
                call.wt[:-1].fill_(0)
            g.replay()
            for call, r in zip(calls, want):
                got = call.result()
                assert np.array_equal(got[0], r[0]) and np.array_equal(got[1], r[1])
            calls[0].run()  # eager work in between
