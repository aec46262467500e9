"""States in 8 bits: codes and scales bit for bit against the formula, the token's read against 64 bits."""
import pytest
import torch

import around64
from around64 import rounded
from plain64 import within

T = {"f32": torch.float32, "bf16": torch.bfloat16}
CODES = [torch.int8, torch.float8_e4m3fn]
SIZES = [(1, 1, 16, 16), (3, 2, 16, 64), (2, 5, 64, 16), (7, 3, 32, 32), (33, 8, 64, 64), (2, 3, 64, 32), (2, 3, 32, 16)]


def state(B, H, D, M, seed=0):
    g = torch.Generator().manual_seed(seed)
    S = torch.randn(B, H, D, M, generator=g) * torch.exp(3 * torch.randn(B, H, D, 1, generator=g))
    S[0, 0, 0] = 0.0
    return S


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("B,H,D,M", SIZES)
def test_pack_and_unpack(cuda, linattn, B, H, D, M, code):
    S = state(B, H, D, M)
    S[-1, -1, -1, :4] = torch.tensor([127.0, 63.5, -62.5, 0.5])  # with the next line: codes half way between two
    S[-1, -1, -1, 4:] = 0.25
    codes, scale = linattn.state_pack(S.to(cuda), code)
    want, ws = around64.pack(S, code)
    assert codes.dtype == code and torch.equal(scale.cpu(), ws)
    assert torch.equal(codes.cpu().view(torch.int8), want.view(torch.int8)) or torch.equal(codes.cpu().float(), want.float())
    back = linattn.state_unpack(codes, scale)
    assert torch.equal(back.cpu(), want.float() * ws[..., None])
    # half a step of the row's largest value at most: of 127 steps, or of e4m3's own (2^-4 relative, 2^-10 / 448 of the
    # largest below its normal range), and the roundings of the scale, the quotient and the product
    top = S.abs().amax(-1, keepdim=True)
    half = top / 254 if code == torch.int8 else torch.maximum(2.0 ** -4 * S.abs(), top * 2.0 ** -10 / 448)
    assert ((back.cpu() - S).abs() <= half * (1 + 2.0 ** -20) + 2.0 ** -22 * S.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_rows_that_are_not_finite_and_tiny_ones(cuda, linattn, code):
    S = state(2, 2, 16, 32, 1)
    S[0, 1, 3, 7], S[0, 1, 4, 8], S[1, 0, 5, 9] = float("nan"), float("inf"), float("-inf")
    S[1, 1, 2] = 0.0
    S[1, 1, 2, 5] = 3e-39   # a scale below the normal range
    S[1, 1, 3] = 1e-45      # a quotient that rounds to nothing
    S[1, 1, 4] = -0.0
    S[1, 1, 6, 0] = 3.0e38
    codes, scale = linattn.state_pack(S.to(cuda), code)
    back = linattn.state_unpack(codes, scale).cpu()
    bad = torch.zeros(2, 2, 16, dtype=torch.bool)
    bad[0, 1, 3] = bad[0, 1, 4] = bad[1, 0, 5] = True
    assert torch.equal(torch.isnan(scale.cpu()), bad)
    assert torch.isnan(back[bad]).all() and torch.isfinite(back[~bad]).all()
    assert float(back[1, 1, 3].abs().max()) == 0.0 and float(back[1, 1, 4].abs().max()) == 0.0
    assert abs(float(back[1, 1, 2, 5]) - 3e-39) < 2e-43 * 127
    assert abs(float(back[1, 1, 6, 0]) / 3.0e38 - 1) < 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("B,Hk,D,M", SIZES)
@pytest.mark.parametrize("r", [1, 3])
def test_step(cuda, linattn, B, Hk, D, M, r, code, dtype):
    g = torch.Generator().manual_seed(2)
    S = state(B, Hk, D, M, 3)
    codes, scale = around64.pack(S, code)
    q, Z = torch.randn(B, Hk * r, D, generator=g).to(T[dtype]), torch.rand(B, Hk, D, generator=g) + 0.5
    Z[-1, -1] = 0.0  # an encoder without states
    y = linattn.cross_step_packed(q.to(cuda), codes.to(cuda), scale.to(cuda), Z.to(cuda))
    want, e = around64.read_packed(q, codes, scale, Z)
    within(y, want, rounded(want, e, dtype), "y")
    assert float(y[-1, -r:].abs().max()) == 0.0
    q[-1, -1], q[0, 0, 3] = float("nan"), float("nan")
    y = linattn.cross_step_packed(q.to(cuda), codes.to(cuda), scale.to(cuda), Z.to(cuda))
    if B * Hk > 1:
        assert float(y[-1, -1].abs().max()) == 0.0 and torch.isnan(y[0, 0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_of_a_cross_attentions_states(cuda, linattn, code):
    """The encoder's S as cross_fwd leaves it, put into 8 bits: the token's read moves by what the codes are off."""
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(s, generator=g).bfloat16().to(cuda) for s in ((2, 4, 5, 64), (2, 2, 700, 64), (2, 2, 700, 64)))
    _, _, S, Z = linattn.cross_fwd(q, k, v)
    codes, scale = linattn.state_pack(S, code)
    qt = q[:, :, 0].contiguous()
    y, full = linattn.cross_step_packed(qt, codes, scale, Z), linattn.cross_step(qt, S, Z)
    f = torch.where(qt > 0, qt.double() + 1, torch.exp(qt.double().clamp(max=0)))
    off = (linattn.state_unpack(codes, scale).double() - S.double()).abs().repeat_interleave(2, 1)
    den = (f * Z.double().repeat_interleave(2, 1)).sum(-1, keepdim=True)
    moved = (f[..., None] * off).sum(-2) / den
    assert ((y.double() - full.double()).abs() <= moved * 1.001 + 2.1 * 2.0 ** -8 * full.double().abs() + 1e-6).all()
    # and through the restored state the same, but for the order of the sums
    near = linattn.cross_step(qt, linattn.state_unpack(codes, scale), Z)
    assert ((y.double() - near.double()).abs() <= 2.1 * 2.0 ** -8 * near.double().abs() + 1e-6).all()


@pytest.mark.gpu
def test_a_parked_decode_state(cuda, linattn):
    """A causal state put away and taken up again: the next token's read is off by what the codes are off."""
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(2, 3, 120, 32, generator=g).to(cuda) for _ in range(3))
    _, _, S, Z = linattn.causal_prefill(q, k, v)
    S2, Z2 = linattn.state_unpack(*linattn.state_pack(S)), Z.clone()
    t = [x[:, :, -1].contiguous() for x in (q, k, v)]
    off = (S2 - S).abs().double()
    a, b = linattn.decode_step(*t, S, Z), linattn.decode_step(*t, S2, Z2)
    f = torch.where(t[0] > 0, t[0].double() + 1, torch.exp(t[0].double().clamp(max=0)))
    den = (f * Z.double()).sum(-1, keepdim=True)
    assert ((a - b).abs().double() <= (f[..., None] * off).sum(-2) / den + 1e-5 * a.abs().double() + 1e-6).all()


@pytest.mark.gpu
def test_offsets_beyond_32_bits(cuda, linattn):
    """More than 2^31 codes: the last heads are those of a call on them alone."""
    B, H, D, M = (1 << 19) + 8, 1, 64, 64
    S = torch.empty(B, H, D, M, device=cuda).normal_()
    codes, scale = linattn.state_pack(S)
    last = linattn.state_pack(S[-8:].contiguous())
    assert torch.equal(codes[-8:], last[0]) and torch.equal(scale[-8:], last[1])
    del S
    assert torch.equal(linattn.state_unpack(codes, scale)[-8:], linattn.state_unpack(*last))
    q, Z = torch.randn(B, H, D, device=cuda), torch.rand(B, H, D, device=cuda) + 1
    y = linattn.cross_step_packed(q, codes, scale, Z)
    assert torch.equal(y[-8:], linattn.cross_step_packed(q[-8:].contiguous(), *last, Z[-8:].contiguous()))


FAKE = 1 << 20


def test_refusals(linattn):
    L, F = linattn.lib(), FAKE
    pack = lambda S=F, c=F, s=F, B=1, H=1, D=16, M=16, f=0: L.la_state_pack(S, c, s, B, H, D, M, f, None)  # noqa: E731
    unpack = lambda c=F, s=F, S=F, B=1, H=1, D=16, M=16, f=0: L.la_state_unpack(c, s, S, B, H, D, M, f, None)  # noqa: E731
    step = lambda q=F, c=F, s=F, Z=F, y=F, B=1, H=2, Hk=1, D=16, M=16, f=0, t=0: L.la_cross_step_packed(q, c, s, Z, y, B, H, Hk, D, M, f, t, None)  # noqa: E731
    for call in (pack, unpack):
        for kw, code in ((dict(S=None), 1), (dict(c=F + 8), 1), (dict(s=None), 1), (dict(B=0), 1), (dict(B=(1 << 20) + 1), 1), (dict(D=48), 2), (dict(M=128), 2),
                         (dict(f=2), 1), (dict(f=-1), 1)):
            assert call(**kw) == code, kw
    for kw, code in ((dict(q=None), 1), (dict(c=F + 4), 1), (dict(s=None), 1), (dict(Z=F + 8), 1), (dict(y=None), 1), (dict(H=3, Hk=2), 1), (dict(D=8), 2), (dict(f=3), 1),
                     (dict(t=5), 1), (dict(B=(1 << 20) + 1, H=1), 1)):
        assert step(**kw) == code, kw


def test_binding_refuses(linattn):
    S = torch.zeros(2, 3, 16, 32)
    codes, scale, q = torch.zeros(2, 3, 16, 32, dtype=torch.int8), torch.zeros(2, 3, 16), torch.zeros(2, 6, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        linattn.state_pack(S)
    with pytest.raises(ValueError, match="CUDA device"):
        linattn.state_unpack(codes, scale)
    with pytest.raises(ValueError, match="CUDA device"):
        linattn.cross_step_packed(q, codes, scale, scale)
    with pytest.raises(TypeError, match="int8 or float8_e4m3fn"):
        linattn.state_pack(S, torch.uint8)
    with pytest.raises(TypeError, match="S: "):
        linattn.state_pack(S.bfloat16())
    with pytest.raises(TypeError, match="int8 or float8_e4m3fn"):
        linattn.state_unpack(S, scale)
    with pytest.raises(ValueError, match="scale: shape"):
        linattn.cross_step_packed(q, codes, scale[:, :2], scale)
    with pytest.raises(ValueError, match="codes: shape"):
        linattn.cross_step_packed(torch.zeros(2, 6, 32), codes, scale, scale)
