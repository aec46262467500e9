"""Plain implementations in 64 bits (torch on the CPU, row by row) of the short
causal convolution, the selective scan and the kernelized cross attention, and
the sizes their roundings are measured against.

Where ``size`` is true a function returns, in place of each output, the sum of
the absolute values of the terms it is a sum of (inputs replaced by their
absolute values; decays, gates and derivatives of the activations are positive
and stay).  An error bound is then a number of roundings times that size.
"""
import math

import torch

F32 = 2.0 ** -24   # half a step, relative
BF16 = 2.0 ** -8


def d64(*ts):
    return [None if t is None else t.detach().double().cpu() for t in ts]


def rows_of(lengths, B, N):
    return [N] * B if lengths is None else [min(max(int(n), 0), N) for n in lengths]


# ------------------------------------------------------------ short convolution

def conv_fwd(x, w, bias, state=None, lengths=None, silu=True):
    """y, the new history, and (for the bounds) pre's size."""
    x, w, bias, state = d64(x, w, bias, state)
    B, N, C = x.shape
    K = w.shape[1]
    y, pre_size = torch.zeros_like(x), torch.zeros_like(x)
    new = torch.zeros(B, K - 1, C, dtype=torch.double) if state is None else state.clone()
    for b, n in enumerate(rows_of(lengths, B, N)):
        hist = list(new[b])
        for t in range(n):
            hist.append(x[b, t])
            taps = torch.stack(hist[-K:])
            pre = (taps * w.t()).sum(0) + (0 if bias is None else bias)
            pre_size[b, t] = (taps.abs() * w.t().abs()).sum(0) + (0 if bias is None else bias.abs())
            y[b, t] = pre / (1 + torch.exp(-pre)) if silu else pre
        new[b] = torch.stack(hist[len(hist) - (K - 1):])
    return y, new, pre_size


def conv_bwd(x, w, bias, dy, lengths=None, silu=True):
    """{dx, dw, db} and {their bounds} in fp32 arithmetic (before a last rounding)."""
    x, w, bias, dy = d64(x, w, bias, dy)
    B, N, C = x.shape
    K = w.shape[1]
    dx, edx = torch.zeros_like(x), torch.zeros_like(x)
    dw, edw = torch.zeros_like(w), torch.zeros_like(w)
    db, edb = torch.zeros(C, dtype=torch.double), torch.zeros(C, dtype=torch.double)
    for b, n in enumerate(rows_of(lengths, B, N)):
        for t in range(n):
            taps = torch.stack([x[b, t - K + 1 + j] if t - K + 1 + j >= 0 else torch.zeros(C, dtype=torch.double) for j in range(K)])
            pre = (taps * w.t()).sum(0) + (0 if bias is None else bias)
            size = (taps.abs() * w.t().abs()).sum(0) + (0 if bias is None else bias.abs())
            s = 1 / (1 + torch.exp(-pre))
            act = s * (1 + pre * (1 - s)) if silu else torch.ones_like(pre)
            g = dy[b, t] * act
            # silu' moves by at most half of pre's error; its own evaluation is ~16 roundings of values up to 1 + |pre|
            eg = dy[b, t].abs() * ((0.5 * (K + 2) * size + 16 * (1 + pre.abs())) * F32 if silu else F32)
            db += g
            edb += eg + 96 * F32 * g.abs()
            for j in range(K):
                dw[:, j] += g * taps[j]
                edw[:, j] += taps[j].abs() * (eg + 96 * F32 * g.abs())  # 32 rows in turn, 8 runs, then the blocks' shares
                r = t - K + 1 + j
                if r >= 0:
                    dx[b, r] += w[:, j] * g
                    edx[b, r] += w[:, j].abs() * (eg + (K + 1) * F32 * g.abs())
    return {"dx": dx, "dw": dw, "db": db}, {"dx": edx, "dw": edw, "db": edb}


# --------------------------------------------------------------- selective scan

def gate(dt, A, bias, lengths):
    dt, A, bias = d64(dt, A, bias)
    z = dt if bias is None else dt + bias
    delta = torch.logaddexp(z, torch.zeros_like(z))
    for b, n in enumerate(rows_of(lengths, dt.shape[0], dt.shape[1])):
        delta[b, n:] = 0.0
    return delta, torch.sigmoid(z), A


def scan(x, dt, A, Bm, Cm, skip=None, dt_bias=None, S=None, lengths=None, dy=None, size=False):
    """{y, S} and, with dy, every gradient."""
    x, Bm, Cm, skip, S, dy = d64(x, Bm, Cm, skip, S, dy)
    delta, sig, A = gate(dt, A, dt_bias, lengths)
    if size:
        x, Bm, Cm, skip, S, dy = [None if t is None else t.abs() for t in (x, Bm, Cm, skip, S, dy)]
    B, N, H, M = x.shape
    G, D = Bm.shape[2:]
    x, Bm, Cm = x.clone(), Bm.clone(), Cm.clone()
    dy = None if dy is None else dy.clone()
    live = torch.zeros(B, N, dtype=torch.double)
    for b, n in enumerate(rows_of(lengths, B, N)):
        live[b, :n] = 1
        for t in (x, Bm, Cm) + (() if dy is None else (dy,)):
            t[b, n:] = 0.0
    Bh, Ch = Bm.repeat_interleave(H // G, 2), Cm.repeat_interleave(H // G, 2)
    a = torch.exp(delta * A)
    St = torch.zeros(B, H, D, M, dtype=torch.double) if S is None else S
    u = delta[..., None] * x
    y, kept = torch.zeros_like(x), []
    for t in range(N):
        kept.append(St)
        St = a[:, t, :, None, None] * St + Bh[:, t, :, :, None] * u[:, t, :, None, :]
        y[:, t] = torch.einsum("bhd,bhdm->bhm", Ch[:, t], St)
    sk = torch.zeros(H, dtype=torch.double) if skip is None else skip
    y = (y + sk[:, None] * x) * live[..., None, None]
    out = {"y": y, "S": St}
    if dy is None:
        return out
    du, dBh, dCh, dl = torch.zeros_like(x), torch.zeros_like(Bh), torch.zeros_like(Ch), torch.zeros_like(delta)
    R = torch.zeros_like(St)
    for t in range(N - 1, -1, -1):
        R = R + Ch[:, t, :, :, None] * dy[:, t, :, None, :]
        dCh[:, t] = torch.einsum("bhdm,bhm->bhd", St, dy[:, t])
        St = kept.pop()
        du[:, t] = torch.einsum("bhd,bhdm->bhm", Bh[:, t], R)
        dBh[:, t] = torch.einsum("bhdm,bhm->bhd", R, u[:, t])
        R = a[:, t, :, None, None] * R
        dl[:, t] = (R * St).sum((2, 3))
    dd = ((du * x).sum(-1) + (A.abs() if size else A) * dl) * live[..., None]
    dz = dd * sig
    out.update(dx=delta[..., None] * du + sk[:, None] * dy, ddt=dz, dA=(delta * dl).sum((0, 1)),
               dBm=dBh.unflatten(2, (G, H // G)).sum(3), dCm=dCh.unflatten(2, (G, H // G)).sum(3),
               dskip=(dy * x).sum((0, 1, 3)), ddt_bias=dz.sum((0, 1)))
    return out


def scan_step_size(dt, A, bias, chunk):
    """Relative error of a chunk's decays in fp32: cum is a sum of up to `chunk` rounded products
    formed by a prefix tree, so each of its 8 levels rounds by half a step of the largest cum."""
    delta, _, A = gate(dt, A, bias, None)
    return 10 * F32 * chunk * float((delta * A.abs()).max()) + 8 * F32


# -------------------------------------------------------------- cross attention

def phi(x):
    return torch.where(x > 0, x + 1, torch.exp(x.clamp(max=0)))


def cross(q, k, v, lengths=None, dout=None, size=False):
    """{out, den, S, Z} and, with dout, {dq, dk, dv}."""
    q, k, v, dout = d64(q, k, v, dout)
    B, H, Nq, D = q.shape
    Hk, Nk, M = k.shape[1], k.shape[2], v.shape[3]
    r = H // Hk
    o = {"out": torch.zeros(B, H, Nq, M, dtype=torch.double), "den": torch.zeros(B, H, Nq, dtype=torch.double),
         "S": torch.zeros(B, Hk, D, M, dtype=torch.double), "Z": torch.zeros(B, Hk, D, dtype=torch.double),
         "dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)}
    ab = (lambda t: t.abs()) if size else (lambda t: t)
    for b, n in enumerate(rows_of(lengths, B, Nk)):
        if n == 0:
            continue
        for h in range(H):
            g = h // r
            fq, fk, vv = phi(q[b, h]), phi(k[b, g, :n]), ab(v[b, g, :n])
            S, Z = fk.t() @ vv, fk.sum(0)
            den = fq @ Z
            out = fq @ S / den[:, None]
            o["out"][b, h], o["den"][b, h], o["S"][b, g], o["Z"][b, g] = out, den, S, Z
            if dout is None:
                continue
            d = ab(dout[b, h]) / den[:, None]
            gam = (d * out).sum(-1) * (1 if size else -1)
            o["dq"][b, h] = (d @ S.t() + gam[:, None] * Z) * torch.where(q[b, h] > 0, 1.0, fq)
            R, rr = fq.t() @ d, fq.t() @ gam
            o["dk"][b, g, :n] += (vv @ R.t() + rr) * torch.where(k[b, g, :n] > 0, 1.0, fk)
            o["dv"][b, g, :n] += fk @ R
    return o


def within(got, want, bound, name):
    """|got - want| <= bound, element by element, and finite."""
    g = got.detach().double().cpu()
    assert g.shape == want.shape, (name, g.shape, want.shape)
    assert torch.isfinite(g).all(), f"{name}: not finite"
    over = (g - want).abs() - bound
    worst = float(over.max()) if over.numel() else -math.inf
    if worst > 0:
        i = int(over.argmax())
        raise AssertionError(f"{name}: {float(g.flatten()[i])!r} for {float(want.flatten()[i])!r}, bound "
                             f"{float(torch.as_tensor(bound).expand_as(g).flatten()[i]):.3e} (entry {i}, "
                             f"{int((over > 0).sum())} of {over.numel()} over)")
