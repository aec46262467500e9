"""Rotary positions against exact angles, within bounds of the roundings of fp32 (around64)."""
import math

import pytest
import torch

import around64
from around64 import rounded
from plain64 import F32, within

T = {"f32": torch.float32, "bf16": torch.bfloat16}


def host_turns(la, R, **kw):
    turns, gain = la.rotary_turns(R, device="cpu", **kw)
    return [t % (1 << 64) for t in turns.tolist()], gain


CASES = [  # B, N, H, Hk, D, R, dtype, pad, lengths
    (1, 1, 1, 0, 2, 2, "f32", 0, None),
    (2, 9, 3, 1, 64, 64, "bf16", 0, None),
    (2, 9, 3, 3, 64, 32, "bf16", 8, [9, 4]),   # half the head, rows of a wider buffer
    (3, 33, 5, 2, 32, 32, "f32", 4, [0, 33, 7]),
    (2, 17, 2, 2, 48, 16, "f32", 0, None),
    (2, 17, 2, 1, 40, 24, "bf16", 3, None),    # rows off the vectors
    (2, 11, 4, 1, 7, 6, "bf16", 0, None),      # odd heads
    (1, 5, 2, 2, 33, 10, "f32", 0, None),
    (1, 3, 1, 1, 1024, 1024, "bf16", 0, None),
    (1, 2, 1, 1, 1023, 1022, "f32", 0, None),
    (1, 400, 40, 8, 64, 64, "bf16", 0, None),  # several heads a thread
]


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("B,N,H,Hk,D,R,dtype,pad,lengths", CASES)
def test_forward_and_inverse(cuda, linattn, B, N, H, Hk, D, R, dtype, pad, lengths, head_major, interleaved):
    g = torch.Generator().manual_seed(B + D)
    t = T[dtype]
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=cuda)
    live = (torch.arange(N)[None, :] < torch.tensor([N] * B if lengths is None else lengths)[:, None])[..., None, None]
    wide = torch.randn(B, N, (H + Hk) * D + pad, generator=g).to(t)
    q = wide[..., :H * D].unflatten(-1, (H, D))
    k = wide[..., H * D:(H + Hk) * D].unflatten(-1, (Hk, D)) if Hk else None
    if head_major:
        dev = lambda v: None if v is None else v.transpose(1, 2).contiguous().to(cuda)  # noqa: E731
        qd, kd = dev(q), dev(k)
    else:
        w = wide.to(cuda)
        qd, kd = w[..., :H * D].unflatten(-1, (H, D)), w[..., H * D:(H + Hk) * D].unflatten(-1, (Hk, D)) if Hk else None
    turns, _ = linattn.rotary_turns(R, device=cuda)
    exact, _ = host_turns(linattn, R)
    start = torch.randint(0, 1 << 20, (B,), generator=g, dtype=torch.int32)
    each = torch.randint(-(1 << 31), (1 << 31) - 1, (B, N), generator=g).to(torch.int32)
    rows = torch.arange(N)
    for positions, at in ((None, rows.expand(B, N)), (start, start[:, None].long() + rows), (each, each.long())):
        for inverse in (False, True):
            call = linattn.rotary_bwd if inverse else linattn.rotary_fwd
            got = call(qd, kd, turns, positions=None if positions is None else positions.to(cuda), gain=1.25, interleaved=interleaved,
                       head_major=head_major, lengths=n)
            for x, y in zip((q, k), got):
                if x is None:
                    assert y is None
                    continue
                want, e = around64.rotary(x, exact, at, 1.25, interleaved, inverse)
                y = y.transpose(1, 2) if head_major else y
                want, e = torch.where(live, want, 0.0), torch.where(live, e, 0.0)
                turned = torch.arange(D) < R
                within(y, want, torch.where(turned, rounded(want, e, dtype), 0.0), "turned")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("head_major", [False, True])
def test_in_place(cuda, linattn, dtype, head_major):
    """In place: the same values, rows past the length and columns past R not touched, neighbours in wider rows neither."""
    g = torch.Generator().manual_seed(3)
    B, N, H, Hk, D, R = 3, 21, 4, 2, 64, 48
    n = torch.tensor([21, 0, 6], dtype=torch.int32, device=cuda)
    wide = torch.randn(B, N, (H + Hk) * D + 24, generator=g).to(T[dtype]).to(cuda)
    views = lambda w: (w[..., 8:8 + H * D].unflatten(-1, (H, D)), w[..., 8 + H * D:8 + (H + Hk) * D].unflatten(-1, (Hk, D)))  # noqa: E731
    q, k = views(wide) if not head_major else (v.transpose(1, 2).contiguous() for v in views(wide))
    turns, _ = linattn.rotary_turns(R, device=cuda)
    before = wide.clone()
    want = linattn.rotary_fwd(q, k, turns, lengths=n, head_major=head_major)
    old = q.clone(), k.clone()
    got = linattn.rotary_fwd(q, k, turns, lengths=n, head_major=head_major, inplace=True)
    assert got[0] is q and got[1] is k
    live = (torch.arange(N, device=cuda)[None, :] < n[:, None])
    live = live[:, None, :, None] if head_major else live[..., None, None]
    for a, b, c in zip(got, want, old):
        assert torch.equal(a, torch.where(live, b, c))
    if not head_major:
        assert torch.equal(wide[..., :8], before[..., :8]) and torch.equal(wide[..., -16:], before[..., -16:])


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_steps_are_the_prompts_rows(cuda, linattn, interleaved):
    g = torch.Generator().manual_seed(4)
    B, N, H, Hk, D = 3, 12, 4, 2, 64
    q, k = torch.randn(B, N, H, D, generator=g).bfloat16().to(cuda), torch.randn(B, N, Hk, D, generator=g).bfloat16().to(cuda)
    turns, gain = linattn.rotary_turns(D, factor=8.0, original=2048, device=cuda)
    start = torch.tensor([0, 77, 1 << 30], dtype=torch.int32, device=cuda)
    how = dict(gain=gain, interleaved=interleaved)
    qa, ka = linattn.rotary_fwd(q, k, turns, positions=start, **how)
    for t in range(N):
        qt, kt = linattn.rotary_fwd(q[:, t], k[:, t], turns, positions=start + t, **how)
        assert torch.equal(qt, qa[:, t]) and torch.equal(kt, ka[:, t])


@pytest.mark.gpu
def test_copied_columns_keep_their_bits(cuda, linattn):
    x = torch.randn(2, 5, 3, 64, device=cuda)
    x[0, 2, 1, 40], x[1, 0, 0, 63] = float("nan"), float("inf")
    y, _ = linattn.rotary_fwd(x, None, linattn.rotary_turns(32, device=cuda)[0])
    assert torch.equal(x[..., 32:].view(torch.int32), y[..., 32:].view(torch.int32))
    assert torch.isfinite(y[..., :32]).all()
    x[1, 3, 2, 5] = float("nan")  # pair 5 is columns 5 and 21
    y, _ = linattn.rotary_fwd(x, None, linattn.rotary_turns(32, device=cuda)[0])
    bad = torch.isnan(y[..., :32])
    assert bad[1, 3, 2, 5] and bad[1, 3, 2, 21] and int(bad.sum()) == 2


@pytest.mark.gpu
def test_scores_depend_on_the_distance(cuda, linattn):
    """q at p against k at p - d: the same product at any p."""
    g = torch.Generator().manual_seed(5)
    D = 64
    q, k = torch.randn(1, 1, 1, D, generator=g).to(cuda), torch.randn(1, 1, 1, D, generator=g).to(cuda)
    turns, _ = linattn.rotary_turns(D, device=cuda)
    size = float((q.abs() * k.abs()).sum())
    at = lambda p: torch.tensor([p], dtype=torch.int32, device=cuda)  # noqa: E731
    score = lambda p: float((linattn.rotary_fwd(q, None, turns, positions=at(p))[0].double() * linattn.rotary_fwd(k, None, turns, positions=at(p - 5))[0].double()).sum())  # noqa: E731
    first = score(5)
    for p in (1000, 1 << 20, (1 << 31) - 1, -(1 << 30)):
        assert abs(score(p) - first) <= 4 * 7 * F32 * 2 * size + 64 * F32 * size


@pytest.mark.gpu
def test_autograd(cuda, linattn):
    g = torch.Generator().manual_seed(6)
    q, k = (torch.randn(2, 9, h, 48, generator=g).to(cuda).requires_grad_(True) for h in (4, 2))
    turns, _ = linattn.rotary_turns(32, device=cuda)
    n = torch.tensor([9, 5], dtype=torch.int32, device=cuda)
    oq, ok = linattn.rotary(q, k, turns, gain=1.5, lengths=n)
    dq, dk = torch.randn_like(oq), torch.randn_like(ok)
    got = torch.autograd.grad((oq, ok), (q, k), (dq, dk))
    want = linattn.rotary_bwd(dq, dk, turns, gain=1.5, lengths=n)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the inverse is the transpose: dy . (y of x) = (dx of dy) . x
    a, b = float((dq.double() * oq.detach().double()).sum()), float((got[0].double() * q.detach().double()).sum())
    assert abs(a - b) <= 32 * F32 * float((dq.abs().double() * oq.detach().abs().double()).sum() + (got[0].abs().double() * q.detach().abs().double()).sum())
    oq, none = linattn.rotary(q, None, turns)
    assert none is None
    (d,) = torch.autograd.grad(oq, q, dq)
    assert torch.equal(d, linattn.rotary_bwd(dq, None, turns)[0])
    oq, ok = linattn.rotary(q, k, turns)
    (d,) = torch.autograd.grad(ok, k, dk)  # only one of the two is used
    assert torch.equal(d, linattn.rotary_bwd(dk, None, turns)[0])


@pytest.mark.gpu
def test_offsets_beyond_32_bits(cuda, linattn):
    N, H, D = (1 << 31) // 1024 + 300, 16, 64
    x = torch.empty(1, N, H, D, dtype=torch.bfloat16, device=cuda).normal_()
    turns, _ = linattn.rotary_turns(D, device=cuda)
    y, _ = linattn.rotary_fwd(x, None, turns)
    last = linattn.rotary_fwd(x[:, -200:].contiguous(), None, turns, positions=torch.tensor([N - 200], dtype=torch.int32, device=cuda))[0]
    assert torch.equal(y[:, -200:], last)
    z, _ = linattn.rotary_fwd(x.view(1, H, N, D), None, turns, head_major=True)
    last = linattn.rotary_fwd(x.view(1, H, N, D)[:, -1:, -200:].contiguous(), None, turns, head_major=True, positions=torch.tensor([N - 200], dtype=torch.int32, device=cuda))[0]
    assert torch.equal(z[:, -1:, -200:], last)


def test_turns(linattn):
    """The frequencies as whole numbers of 2^-64 turns; fast pairs keep theirs, slow ones are stretched."""
    for R, base in ((2, 10000.0), (64, 10000.0), (128, 500000.0), (6, 1.0)):
        got, gain = host_turns(linattn, R, base=base)
        assert gain == 1.0
        for j, t in enumerate(got):
            f = base ** (-2.0 * j / R) / (2 * math.pi)
            assert abs(t / 2.0 ** 64 - f) <= 2.0 ** -50 * f + 2.0 ** -65  # fp64, then a whole number
    plain, _ = host_turns(linattn, 64)
    stretched, gain = host_turns(linattn, 64, factor=4.0)
    assert gain == 1.0 and all(abs(4 * s - p) <= 2.0 ** -40 * p for s, p in zip(stretched, plain))
    ramp, gain = host_turns(linattn, 64, factor=4.0, original=2048)
    assert abs(gain - (0.1 * math.log(4.0) + 1)) < 1e-12
    for s, p in zip(ramp, plain):
        turns = 2048 * p / 2.0 ** 64
        share = min(1.0, max(0.0, (turns - 1) / 31))
        assert abs(s - p * (share + (1 - share) / 4)) <= 2.0 ** -40 * p
    for kw in (dict(dim=3), dict(dim=0), dict(dim=8, base=0.0), dict(dim=8, factor=0.5), dict(dim=8, original=0), dict(dim=8, original=9, fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            linattn.rotary_turns(device="cpu", **kw)


FAKE = 1 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(oq=None), 1), (dict(oq=2 * FAKE + 8), 1), (dict(q=FAKE + 1), 1), (dict(k=None), 1), (dict(ok=None), 1), (dict(Hk=0), 1),
    (dict(oq=FAKE), 1), (dict(turns=None), 1), (dict(turns=FAKE + 4), 1), (dict(positions=FAKE + 2), 1), (dict(lengths=FAKE + 2), 1),
    (dict(gain=float("nan")), 1), (dict(gain=float("inf")), 1), (dict(B=0), 1), (dict(N=0), 1), (dict(H=0), 1), (dict(H=32768, ldq=1 << 30), 1),
    (dict(Hk=-1), 1), (dict(R=0), 1), (dict(R=7), 1), (dict(R=18), 1), (dict(D=1026, ldq=4104, ldk=2052), 2), (dict(ldq=63), 1), (dict(ldk=31), 1),
    (dict(B=1 << 16, N=1 << 16), 1), (dict(dt=2), 1),
])
def test_refusals(linattn, kw, code):
    a = dict(q=FAKE, k=FAKE, oq=2 * FAKE, ok=2 * FAKE, turns=FAKE, positions=None, lengths=None, gain=1.0, B=1, N=4, H=4, Hk=2, D=16, R=16, ldq=64, ldk=32,
             per_row=0, inter=0, major=0, inverse=0, dt=0)
    a.update(kw)
    assert linattn.lib().la_rotary(*a.values(), None) == code


def test_binding_refuses(linattn):
    q, k, t = torch.zeros(2, 5, 4, 16), torch.zeros(2, 5, 2, 16), torch.zeros(8, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA device"):
        linattn.rotary_fwd(q, k, t)
    with pytest.raises(ValueError, match="k: shape"):
        linattn.rotary_fwd(q, k[:, :4], t)
    with pytest.raises(TypeError, match="turns"):
        linattn.rotary_fwd(q, k, t.int())
    with pytest.raises(TypeError, match="positions"):
        linattn.rotary_fwd(q, k, t, positions=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="positions: shape"):
        linattn.rotary_fwd(q, k, t, positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="3 dimensions|4 dimensions"):
        linattn.rotary_fwd(q[:, 0], None, t, head_major=True)
    with pytest.raises(ValueError, match="contiguous"):
        linattn.rotary_fwd(q.transpose(1, 2), None, t, head_major=True)
    with pytest.raises(ValueError, match="dense"):
        linattn.rotary_fwd(q.transpose(1, 2), None, t)
    with pytest.raises(ValueError, match="different tensors"):
        linattn.rotary_fwd(q, q, t, inplace=True)
