"""The short causal convolution against a row-by-row 64-bit implementation.

Bounds: pre is K + 1 roundings of sums no larger than its size; SiLU moves by at
most 1.1 times pre's error and costs a few roundings of its own; a bf16 result is
off by half a bf16 step more.
"""
import pytest
import torch

from plain64 import BF16, F32, conv_bwd, conv_fwd, within

T = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(B, N, C, K, dtype, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(T[dtype])  # noqa: E731
    wide = r(B, N, C + pad)
    return wide, wide[..., :C], r(C, K), r(C), r(B, K - 1, C), r(B, N, C)


def y_bound(y, size, K, dtype):
    e = (1.1 * (K + 1) * size + 16 * y.abs()) * F32
    return e + (BF16 * (y.abs() + e) if dtype == "bf16" else 0)


CASES = [  # B, N, C, K, dtype, pad, lengths
    (1, 1, 8, 4, "f32", 0, None),
    (1, 1, 3, 2, "bf16", 0, None),
    (2, 2, 5, 4, "f32", 0, None),          # fewer rows than taps
    (3, 40, 33, 3, "bf16", 0, [40, 0, 7]),  # channels one by one; an empty sequence
    (2, 131, 64, 4, "bf16", 24, [131, 130]),
    (2, 131, 64, 4, "bf16", 3, None),       # rows off the vectors
    (2, 300, 132, 4, "f32", 4, [300, 257]),  # several row groups, a ragged channel block
    (1, 600, 20, 2, "f32", 0, None),
    (2, 259, 260, 3, "bf16", 60, [1, 259]),
]


def dev_view(wide, C):
    return wide.to("cuda")[..., :C]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,C,K,dtype,pad,lengths", CASES)
@pytest.mark.parametrize("silu", [True, False])
def test_forward(cuda, linattn, B, N, C, K, dtype, pad, lengths, silu):
    wide, x, w, b, s, _ = inputs(B, N, C, K, dtype, pad)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    nd = None if n is None else n.to(cuda)
    y = linattn.short_conv_fwd(dev_view(wide, C), w.to(cuda), b.to(cuda), lengths=nd, silu=silu)
    ref, _, size = conv_fwd(x, w, b, None, lengths, silu)
    within(y, ref, y_bound(ref, size, K, dtype), "y")
    sd = s.to(cuda)
    y = linattn.short_conv_fwd(dev_view(wide, C), w.to(cuda), None, state=sd, lengths=nd, silu=silu)
    ref, new, size = conv_fwd(x, w, None, s, lengths, silu)
    within(y, ref, y_bound(ref, size, K, dtype), "y from a history")
    assert torch.equal(sd.cpu().double(), new), "history"


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,C,K,dtype,pad,lengths", CASES)
def test_backward(cuda, linattn, B, N, C, K, dtype, pad, lengths):
    wide, x, w, b, _, dy = inputs(B, N, C, K, dtype, pad, 1)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=cuda)
    for silu, bias in ((True, b), (False, None)):
        got = linattn.short_conv_bwd(dev_view(wide, C), w.to(cuda), None if bias is None else bias.to(cuda), dy.to(cuda), n, silu)
        want, err = conv_bwd(x, w, bias, dy, lengths, silu)
        for name, g in zip(("dx", "dw", "db"), got):
            if g is None:
                assert bias is None
                continue
            e = err[name]
            within(g, want[name], e + (BF16 * (want[name].abs() + e) if dtype == "bf16" else F32 * want[name].abs()), name)


@pytest.mark.gpu
@pytest.mark.parametrize("B,C,K,dtype,pad", [(1, 1, 2, "f32", 0), (5, 33, 3, "bf16", 7), (300, 64, 4, "bf16", 16), (7, 260, 4, "f32", 4)])
def test_steps_continue_a_prompt(cuda, linattn, B, C, K, dtype, pad):
    """A prompt and then single rows give the whole sequence's rows, bit for bit."""
    wide, x, w, b, s, _ = inputs(B, 9, C, K, dtype, pad, 2)
    xd, wd, bd = dev_view(wide, C), w.to(cuda), b.to(cuda)
    whole_state = s.to(cuda)
    whole = linattn.short_conv_fwd(xd, wd, bd, state=whole_state)
    sd = s.to(cuda)
    part = [linattn.short_conv_fwd(xd[:, :4].contiguous(), wd, bd, state=sd)]
    for t in range(4, 9):
        part.append(linattn.short_conv_step(xd[:, t], wd, bd, sd)[:, None])
    assert torch.equal(torch.cat(part, 1), whole)
    assert torch.equal(sd, whole_state)


@pytest.mark.gpu
def test_offsets_beyond_32_bits(cuda, linattn):
    """More than 2^31 elements in rows of a wider buffer: the last rows equal those of the tail alone."""
    C, K, cut = 2304, 4, 300
    N = (1 << 31) // C + 999
    x = torch.empty(1, N, C + 8, dtype=torch.bfloat16, device=cuda).normal_()[..., :C]
    w, b = torch.randn(C, K, device=cuda).bfloat16(), torch.randn(C, device=cuda).bfloat16()
    y = linattn.short_conv_fwd(x, w, b)
    hist = x[:, -cut - K + 1:-cut].contiguous()
    assert torch.equal(y[:, -cut:], linattn.short_conv_fwd(x[:, -cut:], w, b, state=hist))
    dy = torch.zeros_like(y)
    dy[:, -cut:] = 1.0
    dx, dw, db = linattn.short_conv_bwd(x, w, b, dy)
    part = linattn.short_conv_bwd(x[:, -cut - K:], w, b, dy[:, -cut - K:].contiguous())
    assert torch.equal(dx[:, -cut - K + 1:], part[0][:, 1:]) and float(dx[:, :-cut - K].abs().max()) == 0.0
    # dw and db: the same terms in another order, 96 fp32 roundings of 300 terms below 1.1 x (|x| < 6) each
    # side at most, and the result's own
    for a, c in ((dw, part[1]), (db, part[2])):
        err = (a.double() - c.double()).abs()
        assert (err <= 2.01 * 2.0 ** -8 * c.double().abs() + 2 * 96 * 2.0 ** -24 * cut * 1.1 * 6).all()


@pytest.mark.gpu
def test_padded_rows_are_not_read(cuda, linattn):
    _, x, w, b, s, dy = inputs(2, 50, 32, 4, "bf16")
    n = torch.tensor([0, 13], dtype=torch.int32, device=cuda)
    xd, gd = x.to(cuda).contiguous(), dy.to(cuda)
    clean = [linattn.short_conv_fwd(xd, w.to(cuda), b.to(cuda), lengths=n), *linattn.short_conv_bwd(xd, w.to(cuda), b.to(cuda), gd, n)]
    xd[0], xd[1, 13:], gd[0], gd[1, 13:] = float("nan"), float("inf"), float("nan"), float("-inf")
    state = s.to(cuda)
    dirty = [linattn.short_conv_fwd(xd, w.to(cuda), b.to(cuda), lengths=n), *linattn.short_conv_bwd(xd, w.to(cuda), b.to(cuda), gd, n)]
    for a, c in zip(clean, dirty):
        assert torch.equal(a, c)
    linattn.short_conv_fwd(xd, w.to(cuda), b.to(cuda), state=state, lengths=n)
    assert torch.equal(state[0].cpu(), s[0]) and torch.isfinite(state).all()


@pytest.mark.gpu
def test_gradients_against_differences(cuda, linattn):
    """dx, dw and db along random directions against central differences of the 64-bit forward."""
    _, x, w, b, _, dy = inputs(2, 20, 8, 4, "f32", seed=3)
    leaves = [t.to(cuda).requires_grad_(True) for t in (x.contiguous(), w, b)]
    y = linattn.short_conv(*leaves)
    grads = torch.autograd.grad(y, leaves, dy.to(cuda))
    g = torch.Generator().manual_seed(9)
    for i, d in enumerate(grads):
        v = torch.randn(d.shape, generator=g).double()
        at = lambda h: sum((conv_fwd(*[t.double() + h * v if k == i else t.double() for k, t in enumerate((x, w, b))])[0] * dy.double()).flatten())  # noqa: E731
        fd = float(at(1e-5) - at(-1e-5)) / 2e-5
        size = float((d.double().cpu().abs() * v.abs()).sum())
        assert abs(fd - float((d.double().cpu() * v).sum())) <= 1e-5 * size  # fp32 gradients, differences to ~1e-9


FAKE = 1 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(y=FAKE + 8), 1), (dict(x=FAKE + 2), 1), (dict(bias=FAKE + 4), 1),
    (dict(state=FAKE + 4), 1), (dict(lengths=FAKE + 2), 1), (dict(B=0), 1), (dict(B=65536), 1), (dict(N=0), 1), (dict(C=0), 1),
    (dict(C=65537, ldx=70000), 1), (dict(K=1), 2), (dict(K=5), 2), (dict(K=0), 1), (dict(ldx=7), 1), (dict(dt=3), 1),
])
def test_refusals(linattn, kw, code):
    a = dict(x=FAKE, w=FAKE, bias=None, lengths=None, state=None, y=FAKE, B=1, N=4, C=8, K=4, ldx=8, dt=0)
    a.update(kw)
    L = linattn.lib()
    assert L.la_short_conv_fwd(a["x"], a["w"], a["bias"], a["lengths"], a["state"], a["y"], a["B"], a["N"], a["C"], a["K"], a["ldx"], 1, a["dt"], None) == code


def test_refusals_of_the_other_calls(linattn):
    L, F = linattn.lib(), FAKE
    need = linattn.la_short_conv_workspace_bytes(1, 4, 8, 4, 0)
    assert need > 0 and linattn.la_short_conv_workspace_bytes(1, 4, 8, 5, 0) == 0
    bwd = lambda bias, db, ws, wsb: L.la_short_conv_bwd(F, F, bias, None, F, F, F, db, ws, wsb, 1, 4, 8, 4, 8, 1, 0, None)  # noqa: E731
    assert bwd(None, None, None, 0) == linattn.LA_ERR_WORKSPACE
    assert bwd(None, None, F, need - 1) == linattn.LA_ERR_WORKSPACE
    assert bwd(None, None, F + 8, need) == linattn.LA_ERR_INVALID_ARG
    assert bwd(F, None, F, need) == linattn.LA_ERR_INVALID_ARG
    assert L.la_short_conv_step(F, F, None, None, F, 1, 8, 4, 8, 1, 0, None) == linattn.LA_ERR_INVALID_ARG
    assert L.la_short_conv_step(F, F, None, F, F, (1 << 20) + 1, 8, 4, 8, 1, 0, None) == linattn.LA_ERR_INVALID_ARG


def test_binding_refuses(linattn):
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA device"):
        linattn.short_conv_fwd(x, w)
    with pytest.raises(ValueError, match="w: shape"):
        linattn.short_conv_fwd(x, torch.zeros(9, 4))
    with pytest.raises(TypeError, match="bias"):
        linattn.short_conv_fwd(x, w, torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dense"):
        linattn.short_conv_fwd(torch.zeros(2, 8, 5).transpose(1, 2), w)
    with pytest.raises(ValueError, match="N rows apart"):
        linattn.short_conv_fwd(torch.zeros(5, 2, 8).transpose(0, 1), w)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        linattn.short_conv_fwd(x.half(), w.half())
