"""The gated recurrence at the ends of its decay's range, where it is strong (u = k sigmoid(r) of one to many: a row forgets)
and where a gate is all but closed (u down to 1e-33): every value against 64 bits within bounds that follow the decay a and
beta = sqrt(1 - a^2) in relative terms, so that small ones have to hold as many bits as large ones."""
import pytest
import torch

from around64 import _sig, rounded
from plain64 import F32, d64, within

T = {"f32": torch.float32, "bf16": torch.bfloat16}


class Near:
    """A value in 64 bits and how far off an fp32 computation of it may be; every operation rounds once."""

    def __init__(self, v, e):
        self.v, self.e = v, e

    def _round(self, v, e):
        return Near(v, e + F32 * (v.abs() + e))

    def __mul__(self, o):
        return self._round(self.v * o.v, self.v.abs() * o.e + o.v.abs() * self.e + self.e * o.e)

    def __add__(self, o):
        return self._round(self.v + o.v, self.e + o.e)

    def __sub__(self, o):
        return self._round(self.v - o.v, self.e + o.e)


def gates(r, i, lam, scale):
    """s, g, u, a and beta as Near.  u: k 16 half steps and sigmoid's and a product.  Below one, w = 1 - a is off by as much as u
    and 4 half steps for its polynomial, and a = 1 - w by as much in absolute terms and a rounding.  From one on a is an
    exponential: u's relative error u times, two half steps of the argument u log2(e), and the exponential's 4; w = 1 - a.
    beta = om / sqrt(om + 1.2e-38), om = w (1 + a): half of om's error, 4 half steps of the root, 3 for sums and products, and
    half of what the floor under the root is of om."""
    s, es = _sig(r)
    g, eg = _sig(i)
    soft = torch.logaddexp(lam, torch.zeros_like(lam))
    k = scale * soft
    u = k * s
    eu = 17 * F32 + es  # relative
    a, w = torch.exp(-u), -torch.expm1(-u)
    low = u < 1.001  # at the border the bound of the first form is the wider one
    ew = torch.where(low, w * (eu + 4 * F32), a * (u * (eu + 2 * F32) + 4 * F32) + F32 * w)
    ea = torch.where(low, ew + F32 * a, a * (u * (eu + 2 * F32) + 4 * F32))
    om = -torch.expm1(-2 * u)
    rel = (ew / w + ea / (1 + a) + 2 * F32) / 2 + 7 * F32 + 0.6e-38 / om
    return Near(s, s * es), Near(g, g * eg), Near(u, u * eu), Near(a, ea), Near(torch.sqrt(om), torch.sqrt(om) * rel)


def bounds(x, r, i, lam, scale=8.0, h=None, dy=None):
    """{name: (value, bound before the result's rounding)} of y, the last state h and the gradients.  States and G: as sums of
    terms whose decays were multiplied in another order: four half steps of the terms' sizes a row."""
    x, r, i, lam, h, dy = d64(x, r, i, lam, h, dy)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    B, N, C = x.shape
    s, g, u, a, beta = gates(r, i, lam, scale)
    exact = lambda t: Near(t, torch.zeros_like(t))  # noqa: E731
    put = beta * (g * exact(x))
    state = torch.zeros(B, C, dtype=torch.double) if h is None else h
    size, err = state.abs(), torch.zeros(B, C, dtype=torch.double)
    y, ey, before, ebefore = (torch.zeros_like(x) for _ in range(4))
    for t in range(N):
        before[:, t], ebefore[:, t] = state, err
        at, et = a.v[:, t], a.e[:, t]
        err = (at + et) * err + et * size + put.e[:, t] + 4 * F32 * ((at + et) * size + put.v[:, t].abs())
        state, size = at * state + put.v[:, t], at * size + put.v[:, t].abs()
        y[:, t], ey[:, t] = state, err
    out = {"y": (y, ey), "h": (state, err)}
    if dy is None:
        return out
    G, eG = torch.zeros_like(x), torch.zeros_like(x)
    X, sX, eX = (torch.zeros(B, C, dtype=torch.double) for _ in range(3))
    for t in range(N - 1, -1, -1):
        at, et = a.v[:, t], a.e[:, t]
        G[:, t], eG[:, t], sG = dy[:, t] + X, eX + F32 * (dy[:, t].abs() + sX), dy[:, t].abs() + sX
        X, eX, sX = at * G[:, t], (at + et) * eG[:, t] + et * sG + 4 * F32 * (at + et) * sG, at * sG
    G, before = Near(G, eG), Near(before, ebefore)
    gx = g * exact(x)
    inverse = 1 / beta.v
    inverse = Near(inverse, inverse * (beta.e / beta.v + 4 * F32))
    Q = (a * G) * ((a * gx) * (u * inverse) - u * before)
    one = exact(torch.ones_like(x))
    out["dx"], out["dr"], out["di"] = (G * beta) * g, Q * (one - s), ((G * beta) * gx) * (one - g)
    rho = torch.where(lam < -20, torch.ones_like(lam), torch.sigmoid(lam) / torch.logaddexp(lam, torch.zeros_like(lam)))
    adds = 24 + B * (-(-N // 32)) + 24 + 2 * lam.abs()
    out["dlam"] = Near(rho * Q.v.sum((0, 1)), rho * (Q.e.sum((0, 1)) + adds * F32 * (Q.v.abs() + Q.e).sum((0, 1))))
    return {n: v if isinstance(v, tuple) else (v.v, v.e) for n, v in out.items()}


def inputs(B, N, C, dtype, low, high, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g).to(T[dtype])  # noqa: E731
    lam = (torch.rand(C, generator=g) * (high - low) + low).to(T[dtype])
    return n(B, N, C), n(B, N, C), n(B, N, C), lam, n(B, N, C), torch.randn(B, C, generator=g)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("call", ["step", "prompt"])
def test_one_row_forgets_by_its_decay(cuda, linattn, dtype, call):
    """x = 0: the row returns a h, at u from 0.01 to 80."""
    C = 640
    lam = torch.linspace(-6.5, 10.0, C).to(T[dtype])
    x, r, i, _, _, h = inputs(9, 1, C, dtype, 0, 1, 0)
    x = torch.zeros_like(x)
    hd, a = h.to(cuda), [t.to(cuda) for t in (x, r, i, lam)]
    y = linattn.gated_fwd(*a, h=hd) if call == "prompt" else linattn.gated_step(*(t[:, 0] for t in a[:3]), a[3], hd)[:, None]
    want = bounds(x, r, i, lam, h=h)
    within(hd, *want["h"], "state")
    within(y, want["y"][0], rounded(*want["y"], dtype), "y")
    u = gates(*d64(r, i, lam), 8.0)[2].v
    assert float(u.min()) < 0.02 and float(u.max()) > 60


CASES = [  # B, N, C, dtype, range of lam
    (1, 1, 3, "f32", (0, 4)),
    (2, 60, 64, "f32", (1, 3)),       # one tile
    (2, 60, 70, "bf16", (-1, 2)),
    (3, 300, 72, "f32", (-9, 6)),     # slow and fast channels beside one another
    (2, 300, 33, "f32", (2, 2)),
    (2, 700, 136, "bf16", (-4, 3)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("from_state", [False, True])
@pytest.mark.parametrize("B,N,C,dtype,span", CASES)
def test_strong_decays(cuda, linattn, B, N, C, dtype, span, from_state):
    x, r, i, lam, dy, h = inputs(B, N, C, dtype, *span, 1)
    a = [t.to(cuda) for t in (x, r, i, lam)]
    hd = h.to(cuda) if from_state else None
    y, kept = linattn.gated_fwd(*a, h=hd, keep=True)
    got = linattn.gated_bwd(*a, kept, dy.to(cuda))
    want = bounds(x, r, i, lam, h=h if from_state else None, dy=dy)
    for name, t in zip(("y", "dx", "dr", "di", "dlam"), (y, *got)):
        within(t, want[name][0], rounded(*want[name], dtype), name)
    if from_state:
        within(hd, *want["h"], "state")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_all_but_closed_gates(cuda, linattn, dtype):
    """Every row's u between 1e-33 and 1e-9: y, dx, di and with u / beta dr and dlam go by beta, of 1e-16 to 1e-5."""
    x, r, i, lam, dy, _ = inputs(2, 30, 48, dtype, -60, -24, 2)
    r = (3 * r.float() - 8).clamp(-18, 2).to(r.dtype)
    u = gates(*d64(r, i, lam), 8.0)[2].v
    assert 1e-33 < float(u.min()) < 1e-31 and float(u.max()) < 1e-9
    a = [t.to(cuda) for t in (x, r, i, lam)]
    y, kept = linattn.gated_fwd(*a, keep=True)
    got = linattn.gated_bwd(*a, kept, dy.to(cuda))
    want = bounds(x, r, i, lam, dy=dy)
    for name, t in zip(("y", "dx", "dr", "di", "dlam"), (y, *got)):
        within(t, want[name][0], rounded(*want[name], dtype), name)
