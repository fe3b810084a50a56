"""A layer of FP8 experts on prompts of any length, and with the experts of a checkpoint."""
import numpy as np
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from routed_expert_streaming_amd.runtime import Fp8MoELayer, pack_fp8_expert
from tests import fp8kit
from tests.test_gpu_fp8 import dev, gpu, hidden  # noqa: F401
from tests.test_gpu_fp8_layers import Layer, matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [4096, 4097, 9000])
def test_more_pairs_than_one_call_takes(T):
    """16384 (token, expert) pairs are one call; the last of several may be a single token."""
    layer = Layer(128, 96, 10, 4, True, 5, 3)
    x = hidden(T, T, layer.H).cuda()
    idx, w = layer.layer.route(x)
    out = layer.layer(x)
    assert out.shape == x.shape
    layer.check(x, idx, w, out)


def test_experts_of_a_checkpoint():
    """(codes, scales) of every matrix are taken as they are, whatever made them; mixed with matrices; into a slab on
    the host; and by a layer."""
    H, I, E, k = 288, 160, 6, 2
    rng = np.random.default_rng(8)
    shapes = ((I, H), (I, H), (H, I))
    parts = []  # scales that a quantisation would not give back: no block's largest code is 448's
    for _ in range(E + 1):
        parts.append([(rng.integers(0, 0x70, s).astype(np.uint8) | rng.choice(np.uint8([0, 128]), s),
                       rng.uniform(1e-3, 4e-3, tuple(fp8kit.blocks(n) for n in s)).astype(np.float32)) for s in shapes])
    triples = [[(dev(c).view(torch.float8_e4m3fn) if e % 2 else dev(c), dev(s)) for c, s in p] for e, p in enumerate(parts)]
    for e in range(E):
        want = fp8kit.slab(parts[e])
        assert np.array_equal(pack_fp8_expert(*triples[e]).cpu().numpy(), want)
        host = torch.empty(len(want), dtype=torch.uint8)
        pack_fp8_expert(*triples[e], slab=host)
        assert np.array_equal(host.numpy(), want)
    wide = torch.zeros((I, H + 48), dtype=torch.uint8, device="cuda")  # codes and scales with gaps
    wide[:, 32:32 + H] = triples[0][0][0]
    gaps = torch.zeros((2, 5), device="cuda")
    gaps[:, 1:4] = triples[0][0][1]
    packed = pack_fp8_expert((wide[:, 32:32 + H], gaps[:, 1:4]), *triples[0][1:])
    assert np.array_equal(packed.cpu().numpy(), fp8kit.slab(parts[0]))
    w1 = matrix(1, I, H)
    mixed = pack_fp8_expert(w1, *triples[0][1:]).cpu().numpy()
    assert np.array_equal(mixed, fp8kit.slab([fp8kit.quantise(w1.double().cpu().numpy(), 128)] + parts[0][1:]))

    layer = Layer(H, I, E, k, True, 3, 2)
    layer.layer = Fp8MoELayer(layer.router, triples[:E], k, layer.layer.routing, balance=layer.balance, shared=triples[E])
    layer.parts = parts
    for T in (1, 50):
        x = hidden(T, T, H).cuda()
        idx, w = layer.layer.route(x)
        layer.check(x, idx, w, layer.layer(x))

    good = triples[0]
    slab = torch.full((L.moe_expert_bytes_fp8(H, I),), 7, dtype=torch.uint8, device="cuda")
    codes, scales = good[2]
    for bad in ((codes, scales[:1]), (codes, scales.double()), (codes.view(torch.int8), scales), (codes, scales.cpu()),
                (codes.cpu(), scales.cpu()), (codes[:, :96], scales[:, :1]), good[0]):
        with pytest.raises(ValueError):
            pack_fp8_expert(good[0], good[1], bad, slab=slab)
    with pytest.raises((ValueError, L.MoEError)):  # a rule that only the last matrix would need
        pack_fp8_expert(good[0], good[1], matrix(2, H, I), slab=slab, scale_rule=2)
    assert (slab == 7).all()
