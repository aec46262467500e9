"""The gated recurrence, the layer norm, rotary positions and packed states in 64 bits (torch on the CPU, row by row),
each with the bound that the roundings of an fp32 computation stay under.

Half steps of fp32 (F32 = 2^-24) are counted; a bf16 result is off by half a bf16 step more (``rounded``).  What the
functions used are good for: exp, log1p, division, square root and their hardware approximations 4 half steps each
(2^-22), a sum or product one.  sigmoid: the exponential (4, and 2 |x| at most for its argument x log2(e) in fp32), one
plus it (1) and a quotient, which may be formed from the reciprocal of two sigmoids' product (1 + 4 + 1): 11 + 2 |x|
half steps, relative; one minus it: as many of sigmoid, and one.
"""
import math

import torch

from plain64 import BF16, F32, d64, rows_of


def rounded(want, e, dtype):
    return e + BF16 * (want.abs() + e) if dtype == "bf16" else e + F32 * want.abs()


def _sig(x):
    return 1 / (1 + torch.exp(-x)), (11 + 2 * x.abs()) * F32


def gated(x, r, i, lam, scale=8.0, h=None, lengths=None, dy=None):
    """{name: (value, bound before the result's rounding)} of y, the last state h and, given dy, the gradients.

    u = k s: 16 half steps for k (exp, log1p, the sum, two products) beside sigmoid's.  1 - a: u's and 8, relative, and
    a as far off in absolute terms (u a <= 1 - a), and a rounding.  beta = sqrt((1 - a)(1 + a)) at most as far off as
    1 - a, and 8.  States: one step a row, three for the products of decays they may have been carried by.  Sums from
    the sizes of their terms (a recurrence of the same decays)."""
    x, r, i, lam, h, dy = d64(x, r, i, lam, h, dy)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    B, N, C = x.shape
    soft = torch.logaddexp(lam, torch.zeros_like(lam))
    k = scale * soft
    s, es = _sig(r)
    g, eg = _sig(i)
    u = k * s
    w, a = -torch.expm1(-u), torch.exp(-u)
    beta = torch.sqrt(-torch.expm1(-2 * u))
    eu = 18 * F32 + es
    ea = w * (eu + 8 * F32) + F32
    eb = eu + 16 * F32  # relative, of beta
    put = beta * g * x
    eput = (eb + eg + 3 * F32) * put.abs()
    n = torch.tensor(rows_of(lengths, B, N))
    live = torch.arange(N)[None, :] < n[:, None]
    state = torch.zeros(B, C, dtype=torch.double) if h is None else h
    size, err = state.abs(), torch.zeros(B, C, dtype=torch.double)
    y, ey, before, ebefore, sbefore = (torch.zeros_like(x) for _ in range(5))
    for t in range(N):
        on = live[:, t, None]
        before[:, t], ebefore[:, t], sbefore[:, t] = state, err, size
        new = a[:, t] * state + put[:, t]
        bigger = a[:, t] * size + put[:, t].abs()
        enew = a[:, t] * err + ea[:, t] * size + eput[:, t] + 4 * F32 * bigger
        state, size, err = torch.where(on, new, state), torch.where(on, bigger, size), torch.where(on, enew, err)
        y[:, t], ey[:, t] = torch.where(on, state, 0.0), torch.where(on, err, 0.0)
    out = {"y": (y, ey), "h": (state, err)}
    if dy is None:
        return out
    G, sG, eG = (torch.zeros_like(x) for _ in range(3))
    X, sX, eX = (torch.zeros(B, C, dtype=torch.double) for _ in range(3))
    for t in range(N - 1, -1, -1):
        on = live[:, t, None]
        G[:, t] = torch.where(on, dy[:, t] + X, 0.0)
        sG[:, t] = torch.where(on, dy[:, t].abs() + sX, 0.0)
        eG[:, t] = torch.where(on, eX + F32 * sG[:, t], 0.0)
        X = torch.where(on, a[:, t] * G[:, t], X)
        eX = torch.where(on, a[:, t] * eG[:, t] + ea[:, t] * sG[:, t] + 4 * F32 * a[:, t] * sG[:, t], eX)
        sX = torch.where(on, a[:, t] * sG[:, t], sX)
    gx = g * x
    ratio = torch.where(beta > 0, u / torch.where(beta > 0, beta, 1.0), 0.0)
    dx, dig = G * beta * g, G * beta * gx * (1 - g)
    edx = eG * beta * g + (eb + eg + 4 * F32) * (sG * beta * g)
    edi = eG * (beta * gx * (1 - g)).abs() + sG * (beta * gx).abs() * (g * eg + F32 + (eb + eg + 5 * F32) * (1 - g))
    inner, sinner = a * gx * ratio - u * before, (a * gx * ratio).abs() + u * sbefore
    einner = (a * gx * ratio).abs() * (ea / a.clamp(min=1e-30) + eg + eu + eb + 6 * F32).clamp(max=1) + u * ebefore + u * sbefore * (eu + 3 * F32)
    aG, saG = a * G, a * sG
    eaG = a * eG + ea * sG + 2 * F32 * saG
    Q, sQ = aG * inner, saG * sinner
    eQ = eaG * sinner + saG * einner + 2 * F32 * sQ
    dr, edr = (1 - s) * Q, (1 - s) * eQ + (s * es + 2 * F32) * sQ
    rho = torch.where(lam < -20, torch.ones_like(lam), torch.sigmoid(lam) / soft)
    adds = 24 + B * (-(-N // 32))
    dlam = rho * Q.sum((0, 1))
    edlam = rho * (eQ.sum((0, 1)) + (adds + 24 + 2 * lam.abs()) * F32 * sQ.sum((0, 1)))
    mask = live[..., None]
    cut = lambda v: torch.where(mask, v, 0.0)  # noqa: E731
    return out | {"dx": (cut(dx), cut(edx)), "dr": (cut(dr), cut(edr)), "di": (cut(dig), cut(edi)), "dlam": (dlam, edlam)}


def norm(x, w, b=None, residual=None, groups=1, eps=1e-5, lengths=None, dy=None, ds=None):
    """{name: (value, bound)} of y, s, mean, rstd and, given dy, dx, dw, db.  A group's sums: 64 half steps of the
    terms' sizes (32 terms a thread, then halving).  Sums over rows: one a row and 16."""
    t = x.dtype
    total = x if residual is None else (x.float() + residual.float()).to(t)
    total, w, b, dy, ds = d64(total, w, b, dy, ds)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    shape = total.shape
    B, N = shape[0], shape[1]
    live = torch.arange(N)[None, :] < torch.tensor(rows_of(lengths, B, N))[:, None]
    f = total.unflatten(-1, (groups, -1))
    M = f.shape[-1]
    wg, bg = w.unflatten(-1, (groups, -1)), torch.zeros_like(w).unflatten(-1, (groups, -1)) if b is None else b.unflatten(-1, (groups, -1))
    mean = f.mean(-1, keepdim=True)
    emean = 65 * F32 * f.abs().mean(-1, keepdim=True)
    v = f - mean
    ev = emean + F32 * v.abs()
    var = (v * v).mean(-1, keepdim=True)
    evar = (2 * ev * v.abs() + ev * ev).mean(-1, keepdim=True) + 68 * F32 * var
    rstd = 1 / torch.sqrt(var + eps)
    rel = (evar / (2 * (var + eps)) + 6 * F32).clamp(max=1)
    xh = v * rstd
    exh = ev * rstd * (1 + rel) + xh.abs() * (rel + F32)
    y = xh * wg + bg
    ey = wg.abs() * exh + 3 * F32 * ((xh * wg).abs() + bg.abs())
    on = live[..., None]
    cut = lambda z: torch.where(on, z.flatten(2), 0.0)  # noqa: E731
    out = {"y": (cut(y), cut(ey)), "s": (cut(f), cut(torch.zeros_like(f))), "mean": (cut(mean), cut(emean)), "rstd": (cut(rstd), cut(rstd * rel))}
    if dy is None:
        return out
    d = torch.where(on, dy, 0.0).unflatten(-1, (groups, -1))
    z = d * wg
    m1, m2 = z.mean(-1, keepdim=True), (z * xh).mean(-1, keepdim=True)
    e1 = 66 * F32 * z.abs().mean(-1, keepdim=True)
    e2 = (z.abs() * exh).mean(-1, keepdim=True) + 68 * F32 * (z * xh).abs().mean(-1, keepdim=True)
    inner = z - m1 - xh * m2
    einner = e1 + xh.abs() * e2 + exh * (m2.abs() + e2) + 5 * F32 * (z.abs() + m1.abs() + (xh * m2).abs())
    dx = inner * rstd + (0 if ds is None else ds.unflatten(-1, (groups, -1)))
    edx = einner * rstd * (1 + rel) + inner.abs() * rstd * (rel + 2 * F32) + F32 * dx.abs()
    adds = (B * N + 16) * F32
    dw, db = (d * xh).sum((0, 1)).flatten(), d.sum((0, 1)).flatten()
    edw = ((d.abs() * exh).sum((0, 1)) + adds * (d * xh).abs().sum((0, 1))).flatten()
    edb = adds * d.abs().sum((0, 1)).flatten()
    return out | {"dx": (cut(dx), cut(edx)), "dw": (dw, edw), "db": (db, edb)}


def rotary(x, turns, at, gain=1.0, interleaved=False, inverse=False):
    """(value, bound) of x [..., rows, H, D] turned at the positions `at` [..., rows] (lists of whole numbers).  The
    angle is exact modulo a turn up to 2^-32 turns and its conversion (a half step of pi / 4 at most), sine and cosine
    2 half steps more: 4 half steps of the pair's size each, one for the gain, two for the products."""
    x = x.detach().double().cpu()
    gain = float(torch.tensor(gain, dtype=torch.float32))
    R = 2 * len(turns)
    whole = [[(int(p) * int(t)) % (1 << 64) for t in turns] for p in torch.as_tensor(at).flatten().tolist()]
    angle = torch.tensor([[2 * math.pi * (v / 2.0 ** 64) for v in row] for row in whole], dtype=torch.double)
    angle = angle.view(*torch.as_tensor(at).shape, 1, R // 2) * (-1 if inverse else 1)
    c, s = gain * torch.cos(angle), gain * torch.sin(angle)
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    p, q = a * c - b * s, b * c + a * s
    e = 7 * F32 * abs(gain) * (a.abs() + b.abs())
    y, bound = x.clone(), torch.zeros_like(x)
    for z, first, second in ((y, p, q), (bound, e, e)):
        if interleaved:
            z[..., 0:R:2], z[..., 1:R:2] = first, second
        else:
            z[..., :R // 2], z[..., R // 2:R] = first, second
    return y, bound


def pack(S, code):
    """(codes, scale) in the formula's own fp32 arithmetic (torch on the CPU: IEEE quotients)."""
    S = S.detach().float().cpu()
    top = 127.0 if code == torch.int8 else 448.0
    scale = S.abs().amax(-1) / top
    q = S / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    q = torch.where((scale > 0)[..., None], q, torch.zeros_like(q))
    return (q.round().clamp(-127, 127).to(torch.int8) if code == torch.int8 else q.clamp(-448, 448).to(code)), scale


def read_packed(q, codes, scale, Z):
    """(value, bound) of the token's read: phi 2 |q| + 8 half steps, a weight and its product two, 40 for the sums of
    both, the quotient two."""
    q, scale, Z = d64(q, scale, Z)
    codes = codes.float().double().cpu()
    r = q.shape[1] // codes.shape[1]
    f = torch.where(q > 0, q + 1, torch.exp(q.clamp(max=0)))
    S = (codes * scale[..., None]).repeat_interleave(r, 1)
    z = Z.repeat_interleave(r, 1)
    den = (f * z).sum(-1, keepdim=True)
    y = torch.where(den != 0, (f[..., None] * S).sum(-2) / torch.where(den != 0, den, 1.0), 0.0)
    size = torch.where(den != 0, (f[..., None] * S).abs().sum(-2) / torch.where(den != 0, den, 1.0), 0.0)
    return y, (2 * (2 * float(q.abs().max()) + 8) + 2 + 40 + 70 + 4) * F32 * size
