"""The bf16 cross attention against bounds of what its kernels round and no more (test_cross_values.errors): an
output of zeros, one of the wrong sign, or one from operands of one bf16 term less is outside them, which the
first tests show on the CPU."""
import pytest
import torch

import plain64
from plain64 import within
from test_cross import CASES, inputs, to_cuda
from test_cross_values import bound, errors, run

BF16_CASES = [c for c in CASES if c[7] == "bf16" and c[4] > 1]
FEW = [(1, 2, 1, 40, 1, 64, 64), (2, 4, 2, 130, 2, 32, 64), (1, 2, 2, 7, 3, 64, 16)]  # B, H, Hk, Nq, Nk, D, M


def terms(t, n):
    """t as the sum of n bf16 values."""
    left, total = t.double(), torch.zeros_like(t, dtype=torch.double)
    for _ in range(n):
        part = left.float().bfloat16().double()
        left, total = left - part, total + part
    return total


def worked_out(q, k, v, lengths, dout):
    want, size = (plain64.cross(q, k, v, lengths, dout, size=s) for s in (False, True))
    e = errors(q, k, "bf16", joins=24)  # S: up to 8 steps of a tile, its two accumulators, the records
    return want, {n: bound(n, e, want, size, "bf16") for n in want}


def fails(got, want, b, name):
    with pytest.raises(AssertionError):
        within(got, want, b, name)


@pytest.mark.parametrize("case", BF16_CASES)
def test_bounds_are_below_the_values(case):
    B, H, Hk, Nq, Nk, D, M, dtype, lengths = case
    q, k, v, dout = inputs(B, H, Hk, Nq, Nk, D, M, dtype)
    want, b = worked_out(q, k, v, lengths, dout)
    for n in want:
        assert float(b[n].norm()) < 0.15 * float(want[n].norm()), n
        fails(torch.zeros_like(want[n]), want[n], b[n], n)
        fails(-want[n], want[n], b[n], n)
        # and entry by entry: nearly none would pass as a zero
        at = want[n] != 0
        assert float((b[n][at] < want[n][at].abs()).double().mean()) > 0.85, n


@pytest.mark.parametrize("B,H,Hk,Nq,Nk,D,M,seen", [
    (1, 2, 1, 40, 1, 64, 64, ("S", "dq")),
    (2, 4, 2, 130, 2, 32, 64, ("S", "out", "dq", "dv")),
    (1, 2, 2, 7, 3, 64, 16, ("S", "dq", "dk")),
    (2, 2, 1, 128, 128, 16, 16, ("out", "dq", "dk", "dv")),
])
def test_bounds_refuse_fewer_terms(B, H, Hk, Nq, Nk, D, M, seen):
    """S from two terms of phi(k) where the kernel takes three; out, dq, dk and dv from operands of one term
    where it takes two (where the values cancel enough for a term to show beside their own rounding)."""
    q, k, v, dout = inputs(B, H, Hk, Nq, Nk, D, M, "bf16", 11)
    want, b = worked_out(q, k, v, None, dout)
    r = H // Hk
    fq, fk, vv, g = plain64.phi(q.double()), plain64.phi(k.double()), v.double(), dout.double()
    many = lambda t: t.repeat_interleave(r, 1)  # noqa: E731
    heads = lambda t: t.unflatten(1, (Hk, r)).sum(2)  # noqa: E731
    d = g / want["den"][..., None]
    gam = -(d * want["out"]).sum(-1, keepdim=True)

    def of(n):
        S, R = many(terms(want["S"], n)), terms(heads(terms(fq / want["den"][..., None], n).transpose(-1, -2) @ g), n)
        return {"S": terms(fk, n + 1).transpose(-1, -2) @ vv, "out": (terms(fq, n) @ S) / want["den"][..., None],
                "dq": (d @ S.transpose(-1, -2) + gam * many(want["Z"])[:, :, None]) * torch.where(q > 0, 1.0, fq),
                "dk": (vv @ R.transpose(-1, -2) + heads((gam * fq).sum(2, keepdim=True))) * torch.where(k > 0, 1.0, fk),
                "dv": terms(fk, n) @ R}

    for name, t in of(2).items():
        within(t, want[name], b[name], name)
    for name, t in of(1).items():
        if name in seen:
            fails(t, want[name], b[name], name)


@pytest.mark.gpu
@pytest.mark.parametrize("case", BF16_CASES)
def test_against_pairs(cuda, linattn, case):
    B, H, Hk, Nq, Nk, D, M, dtype, lengths = case
    q, k, v, dout = inputs(B, H, Hk, Nq, Nk, D, M, dtype)
    want, b = worked_out(q, k, v, lengths, dout)
    got = run(linattn, *(t.to(cuda) for t in (q, k, v, dout)), to_cuda(lengths))
    for n in got:
        within(got[n], want[n], b[n], n)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hk,Nq,Nk,D,M", FEW)
def test_few_states(cuda, linattn, B, H, Hk, Nq, Nk, D, M):
    q, k, v, dout = inputs(B, H, Hk, Nq, Nk, D, M, "bf16", 11)
    want, b = worked_out(q, k, v, None, dout)
    got = run(linattn, *(t.to(cuda) for t in (q, k, v, dout)))
    for n in got:
        within(got[n], want[n], b[n], n)
