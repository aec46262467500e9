"""The cross attention's gradients need no `out`: they form dout . out again from S."""
import pytest
import torch

FAKE = 1 << 20


def test_out_may_be_null(linattn):
    """NULL passes the pointer checks (the workspace's comes after them); an unaligned one does not."""
    L, F = linattn.lib(), FAKE
    call = lambda out: L.la_cross_bwd(F, F, F, None, out, F, F, F, F, F, F, F, None, 0, 1, 2, 1, 10, 300, 16, 16, 0, None)  # noqa: E731
    assert call(None) == call(F) == linattn.LA_ERR_WORKSPACE
    assert call(F + 8) == linattn.LA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_without_out(cuda, linattn, dtype):
    g = torch.Generator().manual_seed(3)
    q, k, v, dout = (torch.randn(s, generator=g).to(dtype).to(cuda) for s in ((2, 4, 50, 32), (2, 2, 70, 32), (2, 2, 70, 64), (2, 4, 50, 64)))
    out, den, S, Z = linattn.cross_fwd(q, k, v)
    want = linattn.cross_bwd(q, k, v, None, out, den, S, Z, dout)
    for a, b in zip(linattn.cross_bwd(q, k, v, None, None, den, S, Z, dout), want):
        assert torch.equal(a, b)
    leaves = [t.requires_grad_(True) for t in (q, k, v)]
    y = linattn.cross_linear_attention(*leaves)
    kept = {t.data_ptr() for t in y.grad_fn.saved_tensors if t is not None}
    assert y.data_ptr() not in kept and q.data_ptr() in kept  # the graph does not hold the output
    for a, b in zip(torch.autograd.grad(y, leaves, dout), want):
        assert torch.equal(a, b)
