"""The kernelized cross attention at values the bounds of ordinary inputs do not reach: features of a few
1e-27 (strongly negative q and k) and NaN or infinities in live places.

Bounds, element by element, from what the kernels round, on the sizes of ``plain64.cross(size=True)``:
  phi     2 |x| + 8 half steps: the exponent x log2(e) in fp32, then the exponential
  sums    one half step a summand and 64 for the joins (n rows of a state; on the tensor cores 16 rows a step)
  bf16    phi, S, e phi and R enter products as bf16 terms: three (2^-24) for S, two (2^-16) elsewhere, the
          product of both second terms (2^-16) dropped; every bf16 result is rounded once (half a step of itself)
"""
import pytest
import torch

import plain64
from plain64 import BF16, F32, within

T = {"f32": torch.float32, "bf16": torch.bfloat16}


def errors(q, k, dtype, joins=64):
    """The relative bounds of each output before its last rounding; joins: half steps beside one a row of S and Z."""
    Nq, Nk, r = q.shape[2], k.shape[2], q.shape[1] // k.shape[1]
    two, three = (2.0 ** -16, 2.0 ** -24) if dtype == "bf16" else (0.0, 0.0)
    p = (2 * max(float(q.abs().max()), float(k.abs().max())) + 8) * F32
    e = {"S": p + three + (Nk + joins) * F32, "Z": p + (Nk + joins) * F32}
    e["den"] = p + e["Z"] + 64 * F32
    e["out"] = p + e["S"] + 3 * two + e["den"] + 132 * F32
    t = e["S"] + two + 128 * F32                     # dout S^T
    gam = 2 * e["den"] + p + t + 74 * F32            # -e (e phi(q) . T)
    e["dq"] = max(t + e["den"], gam + e["Z"]) + p + 4 * F32
    R = p + e["den"] + two + (Nq * r + 64) * F32     # sum e phi(q) dout^T
    e["dk"] = max(R + two + 128 * F32, gam + p + (Nq * r + 64) * F32) + p + 4 * F32
    e["dv"] = R + p + 3 * two + 128 * F32
    return e


def bound(name, e, want, size, dtype):
    b = e[name] * size[name]
    return b + BF16 * (want[name].abs() + b) if dtype == "bf16" and name in ("out", "dq", "dk", "dv") else b


def run(la, q, k, v, dout, n=None):
    f = la.cross_fwd(q, k, v, n)
    return dict(zip(("out", "den", "S", "Z", "dq", "dk", "dv"), (*f, *la.cross_bwd(q, k, v, n, *f, dout))))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at_q,at_k,rows", [(-60, 0, slice(None)), (-60, 0, slice(3, 5)), (-25, -25, slice(None)), (0, -40, slice(None))])
@pytest.mark.parametrize("D,M", [(16, 64), (64, 16)])
def test_small_features(cuda, linattn, dtype, at_q, at_k, rows, D, M):
    """den down to 1e-26, whose square is below fp32's range: out and the gradients are of ordinary size."""
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k, v, dout = r(2, 4, 150, D), r(2, 2, 3, D) + at_k, r(2, 2, 3, M), r(2, 4, 150, M)
    q[:, :, rows] += at_q
    q, k, v, dout = (t.to(T[dtype]) for t in (q, k, v, dout))
    want, size = (plain64.cross(q, k, v, None, dout, size=s) for s in (False, True))
    assert float(want["den"].min()) < 1e-15
    got, e = run(linattn, *(t.to(cuda) for t in (q, k, v, dout))), errors(q, k, dtype)
    for name in got:
        within(got[name], want[name], bound(name, e, want, size, dtype), name)


def places(want):
    """Where the 64-bit form is NaN or infinite."""
    return {n: ~torch.isfinite(t) for n, t in want.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which,value", [("q", float("nan")), ("k", float("nan")), ("v", float("nan")), ("dout", float("nan")),
                                         ("q", float("inf")), ("k", float("inf")), ("v", float("-inf")), ("q", float("-inf"))])
def test_live_nan_and_inf(cuda, linattn, dtype, which, value):
    """A NaN or an infinity that counts reaches the outputs it enters and no others; -inf in q alone is phi = 0."""
    g = torch.Generator().manual_seed(6)
    t = [torch.randn(s, generator=g).to(T[dtype]) for s in ((2, 4, 140, 32), (2, 2, 150, 32), (2, 2, 150, 64), (2, 4, 140, 64))]
    clean = run(linattn, *(u.to(cuda) for u in t))
    bad = [u.clone() for u in t]
    bad[("q", "k", "v", "dout").index(which)][1, 1, 130, 7] = value
    got = run(linattn, *(u.to(cuda) for u in bad))
    want = plain64.cross(*bad[:3], None, bad[3])
    at = places(want)
    assert any(m.any() for m in at.values()) == (value != float("-inf") or which != "q")
    for n, m in at.items():
        assert torch.equal(~torch.isfinite(got[n].cpu()), m), n
        # the other batch entry is not touched at all
        assert torch.equal(got[n][0], clean[n][0]), n


@pytest.mark.gpu
def test_a_nan_prompt_and_its_steps_agree(cuda, linattn):
    g = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn(s, generator=g).bfloat16().to(cuda) for s in ((1, 2, 1, 64), (1, 2, 9, 64), (1, 2, 9, 64)))
    q[0, 1, 0, 3] = float("nan")
    out, _, S, Z = linattn.cross_fwd(q, k, v)
    y = linattn.cross_step(q[:, :, 0].contiguous(), S, Z)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(y[0, 1]).all()
    assert torch.isfinite(out[0, 0]).all() and torch.isfinite(y[0, 0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_sequence_without_states_gives_zeros(cuda, linattn, dtype, value):
    """A padded batch entry: no encoder state, and queries and gradients that hold anything."""
    g = torch.Generator().manual_seed(9)
    q, k, v, dout = (torch.randn(s, generator=g).to(T[dtype]).to(cuda) for s in ((2, 4, 140, 32), (2, 2, 150, 32), (2, 2, 150, 64), (2, 4, 140, 64)))
    n = torch.tensor([0, 77], dtype=torch.int32, device=cuda)
    clean = run(linattn, q, k, v, dout, n)
    q[0], dout[0], k[0], v[0] = value, value, value, value
    for name, t in run(linattn, q, k, v, dout, n).items():
        assert float(t[0].abs().max()) == 0.0, name
        assert torch.equal(t[1], clean[name][1]), name
    y = linattn.cross_step(q[:, :, 0].contiguous(), clean["S"], clean["Z"])
    assert float(y[0].abs().max()) == 0.0 and torch.isfinite(y[1]).all()
