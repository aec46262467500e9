"""The kernelized cross attention against a 64-bit implementation over pairs.

Bounds, element by element, on the sizes of ``plain64.cross(size=True)``: in
fp32 a sum over n rows rounds by less than n + 64 half steps of its size (both
sequences' rows are summed, one after the other, in a gradient).  With bf16
inputs phi of one side and the summed states are rounded to bf16 once before a
product and the result once; S is fp32-accurate to two bf16 terms (2^-16), den and
Z are fp32 sums.
"""
import pytest
import torch

import plain64
from plain64 import BF16, F32, within

T = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(B, H, Hk, Nq, Nk, D, M, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(T[dtype])  # noqa: E731
    return r(B, H, Nq, D), r(B, Hk, Nk, D), r(B, Hk, Nk, M), r(B, H, Nq, M)


CASES = [  # B, H, Hk, Nq, Nk, D, M, dtype, lengths
    (1, 1, 1, 1, 1, 16, 16, "f32", None),
    (1, 2, 1, 1, 1, 64, 64, "bf16", None),
    (2, 2, 2, 3, 70, 32, 16, "f32", [70, 0]),
    (2, 4, 2, 65, 130, 64, 64, "f32", [1, 130]),
    (1, 3, 1, 200, 33, 16, 64, "f32", None),
    (2, 2, 2, 129, 257, 64, 64, "bf16", [257, 128]),
    (3, 4, 2, 40, 300, 32, 64, "bf16", [0, 300, 129]),
    (1, 6, 2, 300, 20, 64, 32, "bf16", None),
    (2, 2, 1, 128, 128, 16, 16, "bf16", None),
    (1, 1, 1, 700, 900, 64, 64, "bf16", [899]),
]


def to_cuda(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hk,Nq,Nk,D,M,dtype,lengths", CASES)
def test_against_pairs(cuda, linattn, B, H, Hk, Nq, Nk, D, M, dtype, lengths):
    q, k, v, dout = inputs(B, H, Hk, Nq, Nk, D, M, dtype)
    want, size = plain64.cross(q, k, v, lengths, dout), plain64.cross(q, k, v, lengths, dout, size=True)
    qd, kd, vd, gd = (t.to(cuda) for t in (q, k, v, dout))
    n = to_cuda(lengths)
    out, den, S, Z = linattn.cross_fwd(qd, kd, vd, n)
    dq, dk, dv = linattn.cross_bwd(qd, kd, vd, n, out, den, S, Z, gd)
    linattn.check_device_status()
    f32 = (Nk + 64) * F32
    state = f32 + (2.0 ** -16 if dtype == "bf16" else 0)
    within(S, want["S"], state * size["S"], "S")
    within(Z, want["Z"], f32 * size["Z"], "Z")
    within(den, want["den"], (f32 + 64 * F32) * size["den"], "den")
    # out: phi(q) and S rounded, the result rounded
    half = 3.1 * BF16 if dtype == "bf16" else 0
    within(out, want["out"], (2 * state + 128 * F32 + half) * size["out"], "out")
    # dq: S and (through gamma) out rounded, the result;  dk, dv: phi(q) / den, R, phi(k) rounded, gamma's out, the result
    grad = 4 * state + (Nq * (H // Hk) + 256) * F32 + (4.2 * BF16 if dtype == "bf16" else 0)
    for name, g in (("dq", dq), ("dk", dk), ("dv", dv)):
        within(g, want[name], grad * size[name], name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padded_states_are_not_read(cuda, linattn, dtype):
    q, k, v, dout = (t.to(cuda) for t in inputs(2, 2, 1, 50, 200, 32, 64, dtype, 1))
    n = to_cuda([0, 77])

    def run(k, v):
        f = linattn.cross_fwd(q, k, v, n)
        return [*f, *linattn.cross_bwd(q, k, v, n, *f, dout)]
    clean = run(k, v)
    k, v = k.clone(), v.clone()
    k[0], v[0], k[1, :, 77:], v[1, :, 77:] = float("nan"), float("inf"), float("inf"), float("nan")
    for a, b in zip(clean, run(k, v)):
        assert torch.equal(a, b)
    assert float(clean[0][0].abs().max()) == 0.0 and float(clean[4][0].abs().max()) == 0.0  # out and dq of the empty one


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_offsets_beyond_32_bits(cuda, linattn, dtype):
    """More than 2^31 elements of queries, then of encoder states: the last head's last rows equal those of
    a call on them alone (a row of a product does not depend on the others)."""
    H, D, M, tail, Ne = 8, 32, 32, 128, 150
    N = ((1 << 31) // (H * D) + 3000) // 128 * 128
    last = lambda t: t[:, :, -tail:].contiguous()  # noqa: E731
    k, v = torch.randn(1, H, Ne, D, device=cuda).to(dtype), torch.randn(1, H, Ne, M, device=cuda).to(dtype)
    q = torch.empty(1, H, N, D, dtype=dtype, device=cuda).normal_()
    out, den, S, Z = linattn.cross_fwd(q, k, v)
    few = linattn.cross_fwd(last(q), k, v)
    assert torch.equal(out[:, -1, -tail:], few[0][:, -1]) and torch.equal(den[:, -1, -tail:], few[1][:, -1])
    dout = torch.empty_like(out).normal_()
    dq = linattn.cross_bwd(q, k, v, None, out, den, S, Z, dout)[0]
    few_dq = linattn.cross_bwd(last(q), k, v, None, *few, last(dout))[0]
    assert torch.equal(dq[:, -1, -tail:], few_dq[:, -1])
    del out, den, dout, dq
    # the long tensor as keys, of whose values only the last 100 of the last head are not zero
    vl = torch.zeros(1, H, N, M, dtype=dtype, device=cuda)
    vl[:, -1, -100:] = torch.randn(100, M, device=cuda).to(dtype)
    out, den, S, Z = linattn.cross_fwd(k, q, vl)
    phi = plain64.phi(q[0, -1, -100:].double()).T
    bound = (100 + 64) * F32 + (2.0 ** -16 if dtype == torch.bfloat16 else 0)
    err = (S[0, -1].double() - phi @ vl[0, -1, -100:].double()).abs()
    assert (err <= bound * (phi @ vl[0, -1, -100:].double().abs())).all()
    assert float(S[0, :-1].abs().max()) == 0.0
    # Z: at most 1800 tiles of 64 rows summed in turn, then the blocks' sums
    assert (Z[0, -1].double() / plain64.phi(q[0, -1].double()).sum(0) - 1).abs().max() <= 1800 * 64 * F32
    dout = torch.randn(1, H, Ne, M, device=cuda).to(dtype)
    grads = linattn.cross_bwd(k, q, vl, None, out, den, S, Z, dout)[1:]
    few = linattn.cross_bwd(k, last(q), last(vl), None, out, den, S, Z, dout)[1:]
    for a, b in zip(grads, few):
        assert torch.equal(a[:, -1, -tail:], b[:, -1]) and torch.isfinite(b).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hk,D,M,dtype", [(1, 1, 1, 16, 16, "f32"), (3, 4, 2, 64, 64, "bf16"), (70, 6, 2, 32, 64, "bf16"), (2, 2, 2, 64, 16, "f32")])
def test_step_reads_the_kept_states(cuda, linattn, B, H, Hk, D, M, dtype):
    q, k, v, _ = inputs(B, H, Hk, 1, 90, D, M, dtype, 2)
    lengths = [0] + [90] * (B - 1) if B > 1 else [90]
    _, _, S, Z = linattn.cross_fwd(q.to(cuda), k.to(cuda), v.to(cuda), to_cuda(lengths))
    y = linattn.cross_step(q[:, :, 0].contiguous().to(cuda), S, Z)
    want, size = plain64.cross(q, k, v, lengths), plain64.cross(q, k, v, lengths, size=True)
    e = 2 * ((90 + 64) * F32 + (2.0 ** -16 if dtype == "bf16" else 0)) + 128 * F32 + (BF16 if dtype == "bf16" else 0)
    within(y, want["out"][:, :, 0], e * size["out"][:, :, 0], "y")


@pytest.mark.gpu
def test_gradients_against_differences(cuda, linattn):
    a = inputs(2, 2, 1, 9, 30, 16, 16, "f32", 3)
    q, k, v, dout = a
    n = [30, 11]
    leaves = [t.to(cuda).requires_grad_(True) for t in (q, k, v)]
    grads = torch.autograd.grad(linattn.cross_linear_attention(*leaves, to_cuda(n)), leaves, dout.to(cuda))
    size = plain64.cross(q, k, v, n, dout, size=True)
    g = torch.Generator().manual_seed(9)
    for i, name in enumerate(("dq", "dk", "dv")):
        w = torch.randn(a[i].shape, generator=g).double()
        at = lambda e: float((plain64.cross(*[t.double() + e * w if j == i else t.double() for j, t in enumerate((q, k, v))], n)["out"] * dout.double()).sum())  # noqa: E731
        fd = (at(1e-5) - at(-1e-5)) / 2e-5
        bound = float((size[name] * w.abs()).sum()) * 400 * F32 + 1e-6 * abs(fd)
        # a kink of phi' within a step of 0 is not drawn here
        assert abs(fd - float((grads[i].double().cpu() * w).sum())) <= bound, name


@pytest.mark.gpu
def test_one_state_gives_its_value(cuda, linattn):
    """A single encoder state: out is its value whatever the query, and dq and dk vanish."""
    q, k, v, dout = (t.to(cuda) for t in inputs(1, 2, 2, 70, 1, 64, 64, "f32", 4))
    out, den, S, Z = linattn.cross_fwd(q, k, v)
    dq, dk, dv = linattn.cross_bwd(q, k, v, None, out, den, S, Z, dout)
    within(out, v.expand(-1, -1, 70, -1).double().cpu(), 256 * F32 * 5, "out")
    size = plain64.cross(q.cpu(), k.cpu(), v.cpu(), None, dout.cpu(), size=True)
    within(dq, torch.zeros(dq.shape, dtype=torch.double), 512 * F32 * size["dq"], "dq")
    within(dk, torch.zeros(dk.shape, dtype=torch.double), 512 * F32 * size["dk"], "dk")


FAKE = 1 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=FAKE + 8), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(den=None), 1), (dict(S=None), 1), (dict(Z=FAKE + 4), 1),
    (dict(lengths=FAKE + 2), 1), (dict(Hk=3), 1), (dict(Hk=0), 1), (dict(Nq=0), 1), (dict(Nk=0), 1), (dict(Nk=(1 << 24) + 1), 1),
    (dict(B=65536), 1), (dict(D=48), 2), (dict(M=128), 2), (dict(dt=5), 1), (dict(ws=None), 5), (dict(wsb=8), 5), (dict(ws=FAKE + 8), 1),
])
def test_refusals(linattn, kw, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, lengths=None, out=FAKE, den=FAKE, S=FAKE, Z=FAKE, ws=FAKE, wsb=1 << 40, B=1, H=2, Hk=1, Nq=10, Nk=300, D=16, M=16, dt=0)
    a.update(kw)
    order = ("q", "k", "v", "lengths", "out", "den", "S", "Z", "ws", "wsb", "B", "H", "Hk", "Nq", "Nk", "D", "M", "dt")
    assert linattn.lib().la_cross_fwd(*[a[k] for k in order], None) == code


def test_refusals_of_the_other_calls(linattn):
    L, F = linattn.lib(), FAKE
    need = linattn.la_cross_workspace_bytes(1, 1, 2, 1, 10, 300, 16, 16, 0)
    bwd = lambda dk, wsb: L.la_cross_bwd(F, F, F, None, F, F, F, F, F, F, dk, F, F, wsb, 1, 2, 1, 10, 300, 16, 16, 0, None)  # noqa: E731
    assert bwd(None, need) == 1 and bwd(F, need - 1) == 5
    assert linattn.la_cross_workspace_bytes(0, 1, 3, 2, 10, 300, 16, 16, 0) == 0
    assert L.la_cross_step(F, None, F, F, 1, 2, 1, 16, 16, 0, None) == 1
    assert L.la_cross_step(F, F, F, F, (1 << 20) + 1, 1, 1, 16, 16, 0, None) == 1


def test_binding_refuses(linattn):
    z = torch.zeros
    q, k, v = z(1, 2, 5, 16), z(1, 1, 7, 16), z(1, 1, 7, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        linattn.cross_fwd(q, k, v)
    with pytest.raises(ValueError, match="k: shape"):
        linattn.cross_fwd(q, z(1, 1, 7, 32), v)
    with pytest.raises(TypeError, match="lengths"):
        linattn.cross_fwd(q, k, v, z(1))
    with pytest.raises(ValueError, match="Z: shape"):
        linattn.cross_step(z(1, 2, 16), z(1, 1, 16, 16), z(1, 2, 16))
