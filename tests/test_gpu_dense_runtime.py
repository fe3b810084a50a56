"""The dense MXFP4 operators through the runtime: the views, slabs and pools that its documentation allows."""
import pytest
import torch

from routed_expert_streaming_amd import _lib as L
from routed_expert_streaming_amd.runtime import MxLinear, quantise_mx

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
