"""The gated recurrence against a row-by-row 64-bit implementation, within bounds of the roundings of fp32 (around64)."""
import pytest
import torch

import around64
from around64 import rounded
from plain64 import F32, within

T = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(B, N, C, dtype, pad=0, seed=0, low=-9.0, high=-4.0):
    """x, r and i as slices of one wide row, lam of decays close to one, dy, a state."""
    g = torch.Generator().manual_seed(seed)
    t = T[dtype]
    wide = torch.randn(B, N, 3 * C + pad, generator=g).to(t)
    lam = (torch.rand(C, generator=g) * (high - low) + low).to(t)
    return wide, lam, torch.randn(B, N, C, generator=g).to(t), torch.randn(B, C, generator=g)


def cut(wide, C, dev=None):
    wide = wide if dev is None else wide.to(dev)
    return wide[..., :C], wide[..., C:2 * C], wide[..., 2 * C:3 * C]


CASES = [  # B, N, C, dtype, pad, lengths, range of lam
    (1, 1, 1, "f32", 0, None, (-9, -4)),
    (1, 1, 8, "bf16", 0, None, (-9, -4)),
    (2, 7, 33, "f32", 0, [7, 3], (-9, -4)),        # odd widths: channels one by one
    (3, 64, 64, "bf16", 0, [64, 0, 13], (-9, -4)),  # one tile; an empty sequence
    (2, 65, 66, "f32", 2, None, (-4, 3)),           # a tile and a row; gates that forget
    (2, 130, 130, "bf16", 6, [130, 129], (-9, -4)),
    (2, 200, 65, "bf16", 3, [1, 200], (-6, 0)),
    (1, 700, 70, "f32", 0, None, (-12, -6)),        # a long memory over many tiles
    (3, 513, 20, "bf16", 4, [512, 513, 128], (-9, -4)),
]


def number(lengths, dev):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,C,dtype,pad,lengths,span", CASES)
def test_forward(cuda, linattn, B, N, C, dtype, pad, lengths, span):
    wide, lam, _, h = inputs(B, N, C, dtype, pad, low=span[0], high=span[1])
    n = number(lengths, cuda)
    y = linattn.gated_fwd(*cut(wide, C, cuda), lam.to(cuda), lengths=n)
    want, e = around64.gated(*cut(wide, C), lam, lengths=lengths)["y"]
    within(y, want, rounded(want, e, dtype), "y")
    hd = h.to(cuda)
    y = linattn.gated_fwd(*cut(wide, C, cuda), lam.to(cuda), h=hd, scale=3.3, lengths=n)
    ref = around64.gated(*cut(wide, C), lam, 3.3, h, lengths)
    within(y, ref["y"][0], rounded(*ref["y"], dtype), "y from a state")
    within(hd, ref["h"][0], ref["h"][1], "state")


@pytest.mark.gpu
@pytest.mark.parametrize("from_state", [False, True])
@pytest.mark.parametrize("B,N,C,dtype,pad,lengths,span", CASES)
def test_backward(cuda, linattn, B, N, C, dtype, pad, lengths, span, from_state):
    wide, lam, dy, h = inputs(B, N, C, dtype, pad, 1, *span)
    n, a = number(lengths, cuda), cut(wide, C, cuda)
    y, kept = linattn.gated_fwd(*a, lam.to(cuda), h=h.to(cuda) if from_state else None, lengths=n, keep=True)
    got = linattn.gated_bwd(*a, lam.to(cuda), kept, dy.to(cuda), lengths=n)
    want = around64.gated(*cut(wide, C), lam, 8.0, h if from_state else None, lengths, dy)
    for name, t in zip(("y", "dx", "dr", "di", "dlam"), (y, *got)):
        within(t, want[name][0], rounded(*want[name], dtype), name)


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,C,dtype,lengths", [(1, 9001, 8, "bf16", None), (2, 5000, 6, "f32", [5000, 4231]), (1, 4100, 72, "f32", None)])
def test_states_over_many_tiles(cuda, linattn, B, N, C, dtype, lengths):
    """More tiles than are looked up at once, in both directions."""
    wide, lam, dy, h = inputs(B, N, C, dtype, 0, 10, -13, -7)
    n, a, hd = number(lengths, cuda), cut(wide, C, cuda), h.to(cuda)
    y, kept = linattn.gated_fwd(*a, lam.to(cuda), h=hd, lengths=n, keep=True)
    got = linattn.gated_bwd(*a, lam.to(cuda), kept, dy.to(cuda), lengths=n)
    want = around64.gated(*cut(wide, C), lam, 8.0, h, lengths, dy)
    for name, t in zip(("y", "dx", "dr", "di", "dlam"), (y, *got)):
        within(t, want[name][0], rounded(*want[name], dtype), name)
    within(hd, *want["h"], "state")


@pytest.mark.gpu
@pytest.mark.parametrize("B,C,dtype,pad", [(1, 1, "f32", 0), (5, 33, "bf16", 7), (300, 64, "bf16", 16), (7, 1030, "f32", 4)])
def test_steps_continue_a_prompt(cuda, linattn, B, C, dtype, pad):
    wide, lam, _, h = inputs(B, 90, C, dtype, pad, 2)
    x, r, i = cut(wide, C, cuda)
    hd, ld = h.to(cuda), lam.to(cuda)
    part = [linattn.gated_fwd(x[:, :80].contiguous(), r[:, :80].contiguous(), i[:, :80].contiguous(), ld, h=hd)]
    for t in range(80, 90):
        part.append(linattn.gated_step(x[:, t], r[:, t], i[:, t], ld, hd)[:, None])
    want = around64.gated(*cut(wide, C), lam, 8.0, h)
    within(torch.cat(part, 1), want["y"][0], rounded(*want["y"], dtype), "y")
    within(hd, want["h"][0], want["h"][1], "state")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_closed_and_open_gates(cuda, linattn, dtype):
    """r far out on both sides, lam from a rate of 1e-26 to one that forgets at once: finite, and what the formulas say."""
    wide, lam, dy, _ = inputs(2, 150, 64, dtype, 0, 3)
    x, r, i = (t.clone() for t in cut(wide, 64))
    r[0, ::3], r[1, ::2], i[0, ::5] = -300.0, 90.0, -200.0
    lam[:16], lam[16:32] = -60.0, 40.0
    a = [t.to(cuda) for t in (x, r, i, lam)]
    y, kept = linattn.gated_fwd(*a, keep=True)
    got = linattn.gated_bwd(*a, kept, dy.to(cuda))
    want = around64.gated(x, r, i, lam, dy=dy)
    # below 2^-126 the hardware's results are zero: 1e-18 covers the roots of such values
    for name, t in zip(("y", "dx", "dr", "di", "dlam"), (y, *got)):
        within(t, want[name][0], rounded(*want[name], dtype) + 1e-18 * (1 + dy.abs().double().sum()), name)


@pytest.mark.gpu
def test_padded_rows_are_not_read(cuda, linattn):
    wide, lam, dy, h = inputs(2, 150, 32, "bf16", 0, 4)
    n = torch.tensor([0, 70], dtype=torch.int32, device=cuda)

    def run(wide, dy):
        a = cut(wide, 32)
        hd = h.to(cuda)
        y, kept = linattn.gated_fwd(*a, lam.to(cuda), lengths=n, keep=True)
        return [y, *linattn.gated_bwd(*a, lam.to(cuda), kept, dy, lengths=n), linattn.gated_fwd(*a, lam.to(cuda), h=hd, lengths=n), hd]

    wd, gd = wide.to(cuda), dy.to(cuda)
    clean = run(wd, gd)
    wd[0], wd[1, 70:], gd[0], gd[1, 70:] = float("nan"), float("inf"), float("nan"), float("-inf")
    for a, b in zip(clean, run(wd, gd)):
        assert torch.equal(a, b)
    assert torch.equal(clean[-1][0].cpu(), h[0])
    for t in clean[:4]:
        assert float(t[0].abs().max()) == 0.0 and float(t[1, 70:].abs().max()) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_live_nan(cuda, linattn, dtype, which):
    """A NaN at a row reaches its channel from that row on, and with the gradients its channel up to and beyond it."""
    wide, lam, dy, _ = inputs(2, 200, 32, dtype, 0, 5)
    a = [t.to(cuda).contiguous() for t in cut(wide, 32)]
    clean = linattn.gated_fwd(*a, lam.to(cuda))
    a[which][1, 130, 5] = float("nan")
    y, kept = linattn.gated_fwd(*a, lam.to(cuda), keep=True)
    bad = torch.zeros(2, 200, 32, dtype=torch.bool, device=cuda)
    bad[1, 130:, 5] = True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], clean[~bad])
    for t in linattn.gated_bwd(*a, lam.to(cuda), kept, dy.to(cuda)):
        t = t if t.dim() == 3 else t[None, None]
        other = [c for c in range(32) if c != 5]
        assert torch.isfinite(t[..., other]).all() and torch.isfinite(t[0, :, other] if t.shape[0] > 1 else t[..., other]).all()


@pytest.mark.gpu
def test_repeats_itself(cuda, linattn):
    wide, lam, dy, _ = inputs(3, 1500, 200, "bf16", 0, 6)
    a = cut(wide, 200, cuda)

    def run():
        y, kept = linattn.gated_fwd(*a, lam.to(cuda), keep=True)
        return [y, *linattn.gated_bwd(*a, lam.to(cuda), kept, dy.to(cuda))]

    first = run()
    for _ in range(20):
        for p, q in zip(first, run()):
            assert torch.equal(p, q)


@pytest.mark.gpu
def test_offsets_beyond_32_bits(cuda, linattn):
    """More than 2^31 elements: the last rows equal those of the tail, whose decays forget what came before."""
    C, cut_at = 2048, 600
    N = (1 << 31) // C + 777
    x = torch.empty(1, N, C, dtype=torch.bfloat16, device=cuda).normal_()
    lam = torch.full((C,), 2.0, dtype=torch.bfloat16, device=cuda)
    h = torch.zeros(1, C, device=cuda)
    y = linattn.gated_fwd(x, x, x, lam, h=h)
    tail = x[:, -cut_at:].contiguous()
    h2 = torch.zeros(1, C, device=cuda)
    y2 = linattn.gated_fwd(tail, tail, tail, lam, h=h2)
    # decays below 0.85 a row (r > -3.4 in most rows): 300 rows on, nothing is left; the rest is order of roundings
    assert float((h - h2).abs().max()) < 1e-5
    d = (y[:, -300:].float() - y2[:, -300:].float()).abs()
    assert (d <= 2 * 2.0 ** -8 * y2[:, -300:].float().abs() + 1e-5).all()
    del y, y2, h
    dy = torch.zeros_like(x)
    dy[:, -cut_at:] = 1.0
    kept = linattn.gated_fwd(x, x, x, lam, keep=True)[1]
    got = linattn.gated_bwd(x, x, x, lam, kept, dy)
    kept = linattn.gated_fwd(tail, tail, tail, lam, keep=True)[1]
    want = linattn.gated_bwd(tail, tail, tail, lam, kept, dy[:, -cut_at:].contiguous())
    for a, b in zip(got[:3], want[:3]):
        d = (a[:, -300:].float() - b[:, -300:].float()).abs()
        assert (d <= 2 * 2.0 ** -8 * b[:, -300:].float().abs() + 1e-5).all()
        assert float(a[:, :1000].abs().max()) < 1e-5


@pytest.mark.gpu
def test_gradients_against_differences(cuda, linattn):
    wide, lam, dy, _ = inputs(2, 70, 6, "f32", 0, 7, -6, -1)
    leaves = [t.contiguous().to(cuda).requires_grad_(True) for t in (*cut(wide, 6), lam)]
    grads = torch.autograd.grad(linattn.gated_recurrence(*leaves), leaves, dy.to(cuda))
    g = torch.Generator().manual_seed(9)
    host = [t.detach().cpu().double() for t in leaves]
    for j, d in enumerate(grads):
        v = torch.randn(d.shape, generator=g).double()
        at = lambda e: float((around64.gated(*[t + e * v if k == j else t for k, t in enumerate(host)])["y"][0] * dy.double()).sum())  # noqa: E731
        fd = (at(1e-5) - at(-1e-5)) / 2e-5
        size = float((d.double().cpu().abs() * v.abs()).sum())
        assert abs(fd - float((d.double().cpu() * v).sum())) <= 2e-5 * size  # fp32 gradients, differences to ~1e-9


FAKE = 1 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(r=None), 1), (dict(i=None), 1), (dict(lam=None), 1), (dict(y=None), 1), (dict(y=FAKE + 8), 1), (dict(x=FAKE + 2), 1),
    (dict(lam=FAKE + 4), 1), (dict(h=FAKE + 4), 1), (dict(kept=FAKE + 8), 1), (dict(lengths=FAKE + 2), 1), (dict(B=0), 1), (dict(B=65536), 1),
    (dict(N=0), 1), (dict(N=(1 << 24) + 1), 1), (dict(C=0), 1), (dict(C=65537, ldx=70000, ldr=70000, ldi=70000), 1), (dict(ldx=7), 1),
    (dict(ldr=7), 1), (dict(ldi=7), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(dt=2), 1),
    (dict(N=5000), 5), (dict(N=5000, ws=FAKE, wsb=16), 5), (dict(N=5000, ws=FAKE + 8, wsb=1 << 30), 1),
])
def test_refusals(linattn, kw, code):
    a = dict(x=FAKE, r=FAKE, i=FAKE, lam=FAKE, lengths=None, h=None, kept=None, y=FAKE, ws=None, wsb=0, B=1, N=4, C=8, ldx=8, ldr=8, ldi=8, scale=8.0, dt=0)
    a.update(kw)
    L = linattn.lib()
    assert L.la_gated_fwd(a["x"], a["r"], a["i"], a["lam"], a["lengths"], a["h"], a["kept"], a["y"], a["ws"], a["wsb"], a["B"], a["N"], a["C"],
                          a["ldx"], a["ldr"], a["ldi"], a["scale"], a["dt"], None) == code


def test_refusals_of_the_other_calls(linattn):
    L, F = linattn.lib(), FAKE
    need = linattn.la_gated_workspace_bytes(1, 1, 4, 8, 0)
    assert need > 0 and linattn.la_gated_workspace_bytes(1, 1, 4, 0, 0) == 0 and linattn.la_gated_kept_bytes(0, 4, 8, 0) == 0
    bwd = lambda kept, ws, wsb: L.la_gated_bwd(F, F, F, F, None, kept, F, F, F, F, F, ws, wsb, 1, 4, 8, 8, 8, 8, 8.0, 0, None)  # noqa: E731
    assert bwd(None, F, need) == linattn.LA_ERR_INVALID_ARG
    assert bwd(F, None, 0) == linattn.LA_ERR_WORKSPACE
    assert bwd(F, F, need - 1) == linattn.LA_ERR_WORKSPACE
    assert bwd(F, F + 8, need) == linattn.LA_ERR_INVALID_ARG
    step = lambda h, B: L.la_gated_step(F, F, F, F, h, F, B, 8, 8, 8, 8, 8.0, 0, None)  # noqa: E731
    assert step(None, 1) == linattn.LA_ERR_INVALID_ARG
    assert step(F, (1 << 20) + 1) == linattn.LA_ERR_INVALID_ARG


def test_binding_refuses(linattn):
    x, lam = torch.zeros(2, 5, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA device"):
        linattn.gated_fwd(x, x, x, lam)
    with pytest.raises(ValueError, match="lam: shape"):
        linattn.gated_fwd(x, x, x, torch.zeros(9))
    with pytest.raises(ValueError, match="r: shape"):
        linattn.gated_fwd(x, x[:, :4], x, lam)
    with pytest.raises(TypeError, match="i: "):
        linattn.gated_fwd(x, x, x.bfloat16(), lam)
    with pytest.raises(ValueError, match="dense"):
        linattn.gated_fwd(torch.zeros(2, 8, 5).transpose(1, 2), x, x, lam)
    with pytest.raises(ValueError, match="scale"):
        linattn.gated_fwd(x, x, x, lam, scale=-1.0)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        linattn.gated_fwd(x.half(), x.half(), x.half(), lam.half())
    with pytest.raises(ValueError, match="h: shape"):
        linattn.gated_fwd(x, x, x, lam, h=torch.zeros(2, 7))
