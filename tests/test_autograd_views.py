"""What autograd hands the layer's functions: gradients that are views, at any address."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def functions(la, dtype, device):
    """Each function with leaves whose output has an odd number of rows."""
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(s, generator=g).to(dtype).to(device).requires_grad_(True)  # noqa: E731
    x, dt, A, b, c = r(1, 3, 2, 16), r(1, 3, 2), (-torch.ones(2, dtype=dtype, device=device)).requires_grad_(True), r(1, 3, 1, 16), r(1, 3, 1, 16)
    return {
        "short_conv": (la.short_conv, [r(1, 3, 5), r(5, 3)]),
        "selective_scan": (la.selective_scan, [x, dt, A, b, c]),
        "cross_linear_attention": (la.cross_linear_attention, [r(1, 2, 5, 16), r(1, 1, 7, 16), r(1, 1, 7, 16)]),
    }


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", ["short_conv", "selective_scan", "cross_linear_attention"])
def test_gradient_at_an_odd_address(cuda, linattn, name, dtype):
    """A result behind others in one vector: its gradient is a dense view that starts one element in."""
    f, leaves = functions(linattn, dtype, cuda)[name]
    y = f(*leaves)
    d = torch.randn(y.numel() + 1, device=cuda).to(dtype)
    want = torch.autograd.grad(f(*leaves), leaves, d[1:].clone().view(y.shape))
    got = torch.autograd.grad(torch.cat([torch.zeros(1, dtype=dtype, device=cuda), y.flatten()]), leaves, d)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
