"""The bf16 scan's gate gradients and final state against bounds of what its kernels round and no more.

ddt, dA and ddt_bias are sums that cancel far below their terms, so the kernels form them from fp32 scores and
from carried states in two bf16 terms.  ``gate_bounds`` follows those sums chunk by chunk (128 rows) in 64 bits, the
absolute values of the terms beside a bound of each one's error:
  gate      delta: 6 + |z| half steps (z = dt + bias rounded, exponential, logarithm);
  decays    an exponent's rounding: 9 + |z| half steps of itself (delta, two products), 8 of its 32-row blocks' prefix
            sums and 12 of the chunk's where it spans blocks; 24 for the exponentials and their products;
  products  16 rows a step of the tensor cores, 10.5 half steps each (16 truncations below the last bit, one of
            the sum): 42 for 64 columns, 84 for 128 rows;
  states    two bf16 terms where they are summed and two where they are kept, 2^-16 each; 4 half steps a chunk;
  sums      as many half steps as a sum is deep;
and one rounding of the result to bf16.  Tests on the CPU show that zeros, flipped signs, states of one term and
missing pairs are outside them, and a final state from two terms where the kernel takes three.
"""
import pytest
import torch

import plain64
from plain64 import BF16, F32, within
from test_scan import CASES, PARAMS, inputs, place, to_cuda

TWO, CH = 2.0 ** -16, 128
NAMES = ("ddt", "dA", "ddt_bias")
BF16_CASES = [(*c, 1.0) for c in CASES if c[6] == "bf16"] + [  # and how fast A decays
    (1, 40, 2, 1, 32, 64, "bf16", None, 1.0), (1, 1200, 2, 1, 16, 32, "bf16", [1100], 1.0), (1, 300, 40, 1, 16, 16, "bf16", None, 1.0),
    (1, 500, 3, 1, 64, 64, "bf16", None, 0.02), (2, 700, 2, 1, 16, 32, "bf16", [640, 700], 0.02)]


def chunks(x, dt, A, Bm, Cm, skip, dt_bias, lengths, dy):
    """[batch entry][head] lists of the chunks with their states, and sigma(z), delta and |z|'s largest."""
    delta, sig, A = plain64.gate(dt, A, dt_bias, lengths)
    z = float((dt.double() + dt_bias.double()).abs().max())
    x, Bm, Cm, dy = (t.clone() for t in plain64.d64(x, Bm, Cm, dy))
    B, N, H, M = x.shape
    r = H // Bm.shape[2]
    for b, n in enumerate(plain64.rows_of(lengths, B, N)):
        for t in (x, Bm, Cm, dy):
            t[b, n:] = 0
    found = []
    for b in range(B):
        found.append([])
        for h in range(H):
            parts = [Chunk(*(t[b, i:i + CH] for t in (x[:, :, h], Bm[:, :, h // r], Cm[:, :, h // r], dy[:, :, h])),
                           delta[b, i:i + CH, h], float(A[h]), z) for i in range(0, N, CH)]
            S = torch.zeros(3, Bm.shape[3], M, dtype=torch.double)  # a state, its terms' absolute values, its error
            for c in parts:
                c.S, S = S, c.carry(S, c.F)
            R = torch.zeros_like(S)
            for c in reversed(parts):
                c.R, R = R, c.carry(R, c.E)
            found[b].append(parts)
    return found, sig, delta, z


def rows_from(found, f):
    """f(chunk) of every chunk as tensors [B, N, H]."""
    cols = [[[f(c) for c in parts] for parts in heads] for heads in found]
    return [torch.stack([torch.stack([torch.cat([c[k] for c in parts]) for parts in heads], 1) for heads in cols]) for k in range(len(cols[0][0][0]))]


def gate_bounds(*args):
    """{ddt, dA, ddt_bias}: bounds of the kernels' errors before the last rounding."""
    found, sig, delta, z = chunks(*args)
    exu, xu, edl, dl = rows_from(found, Chunk.bounds)
    A = args[2].double().abs()
    last = (24 + delta.shape[1] / CH) * F32  # the sums over rows, chunks and batch entries
    dz = sig * (xu + A * dl)
    edz = sig * (exu + A * edl) + (14 + z) * F32 * dz
    return {"ddt": edz, "dA": (delta * (edl + ((8 + z) * F32 + last) * dl)).sum((0, 1)), "ddt_bias": (edz + last * dz).sum((0, 1))}


def gate_values(args, kept, pairs):
    """{ddt, dA, ddt_bias} by the kernels' sums, in 64 bits, with what `kept` makes of the carried states and `pairs` of the pair sums."""
    found, sig, delta, _ = chunks(*args)
    xu, dl = rows_from(found, lambda c: c.values(kept, pairs))
    ddt = sig * (xu + args[2].double() * dl)
    return {"ddt": ddt, "dA": (delta * dl).sum((0, 1)), "ddt_bias": ddt.sum((0, 1))}


class Chunk:
    """One chunk and head.  (value, relative error) pairs for the decays; (value, error) for sums."""

    def __init__(self, x, B, C, dy, delta, A, z):
        self.x, self.B, self.C, self.dy, self.delta, self.A, self.z = x, B, C, dy, delta, A, z
        n = len(delta)
        cum = torch.cumsum(delta * abs(A), 0)
        block = torch.arange(n) // 32
        wp = cum - torch.where(block > 0, cum[(32 * block - 1).clamp(min=0)], 0.0)  # of the row's block alone
        tot, tb = cum[-1], wp.max()

        def decay(d, prefix, far):  # exp(-d)
            return torch.exp(-d), F32 * ((9 + z) * d + 8 * prefix + 12 * tot * far + 24)
        self.start, self.end, self.down = decay(cum, wp, 1.0), decay(tot - cum, wp + tb, 1.0), decay(tot, tb, 1.0)
        W, eW = decay((cum[:, None] - cum[None, :]).clamp(min=0), wp[:, None] + wp[None, :] + tb, (block[:, None] - block[None, :] > 1).double())
        a, e = C @ B.t(), dy @ x.t()  # [i, j]
        ea, ee = (42 * F32 * (u.abs() @ v.abs().t()) for u, v in ((C, B), (dy, x)))
        low = torch.ones(n, n, dtype=torch.bool).tril(-1)
        self.G = torch.where(low, W * a * e, 0.0)  # without delta
        self.eG = torch.where(low, W * (ea * e.abs() + a.abs() * ee), 0.0) + self.G.abs() * (eW + 4 * F32)
        self.self_ = (a * e).diagonal(), (ea * e.abs() + a.abs() * ee).diagonal() + 2 * F32 * (a * e).diagonal().abs()

        def own(rows, cols, f, ef):
            v, s = rows.t() @ (f[:, None] * cols), rows.abs().t() @ (f[:, None] * cols.abs())
            return torch.stack([v, s, rows.abs().t() @ ((f * (ef + TWO + (8 + z) * F32))[:, None] * cols.abs()) + 84 * F32 * s])
        self.F, self.E = own(B, x, delta * self.end[0], self.end[1]), own(C, dy, *self.start)

    def carry(self, S, F):
        (v, s, e), (f, ef) = S, self.down
        return torch.stack([f * v + F[0], f * s + F[1], f * (e + v.abs() * ef) + F[2] + 4 * F32 * (f * s + F[1])])

    def read(self, f, T, rows, cols):
        """f_i rows_i . (T cols_i) and its error: T kept in two terms, a product over M and one over D."""
        at = lambda T: torch.einsum("id,dm,im->i", rows.abs(), T, cols.abs())  # noqa: E731
        v = f[0] * torch.einsum("id,dm,im->i", rows, T[0], cols)
        return v, v.abs() * (f[1] + 4 * F32) + f[0] * (at(T[2] + TWO * T[0].abs()) + 62 * F32 * at(T[0].abs()))

    def values(self, kept, pairs):
        """x . du and dl by row (the pairs of dl as differences of row and column sums)."""
        S, R, G, delta = [kept(self.S[0])], [kept(self.R[0])], pairs(self.G), self.delta
        v, w = (f[0] * torch.einsum("id,dm,im->i", a, T[0], b) for f, a, T, b in ((self.start, self.C, S, self.dy), (self.end, self.B, R, self.x)))
        net = v + (G * delta).sum(1) - delta * G.sum(0)
        return G.sum(0) + self.self_[0] + w, suffix(net) + before(delta * w) + self.down[0] * (S[0] * R[0]).sum()

    def bounds(self):
        """By row: the error of x . du and its size, the error of dl and its size (sizes without the cancellation between
        their few parts)."""
        delta, z = self.delta, self.z
        (v, ev), (w, ew) = self.read(self.start, self.S, self.C, self.dy), self.read(self.end, self.R, self.B, self.x)
        S, R, (f, ef) = self.S, self.R, self.down
        sr = f * (S[0] * R[0]).sum()
        k = lambda T: T[2] + TWO * T[0].abs()  # noqa: E731
        esr = f * (k(S) * R[0].abs() + S[0].abs() * k(R) + 40 * F32 * (S[0] * R[0]).abs()).sum() + sr.abs() * ef
        # The pairs that span row t, i >= t > j.  A pair's own error enters its row's sum and its column's alike and
        # leaves with it where both are past t; what the two sums' own roundings (36 half steps) leave does not.
        over = lambda G: torch.cat([torch.zeros(len(delta), 1, dtype=torch.double), torch.cumsum(suffix(G), 1)[:, :-1]], 1).diagonal()  # noqa: E731
        span, espan = over(self.G * delta), over((self.eG + (6 + z) * F32 * self.G.abs()) * delta)
        row, col = (self.G.abs() * delta).sum(1), self.G.abs().sum(0)
        net = v + (self.G * delta).sum(1) - delta * self.G.sum(0)
        ww, eww = delta * w, delta * (ew + (8 + z) * F32 * w.abs())
        edl = espan + suffix(ev + 36 * F32 * (v.abs() + row + delta * col) + 12 * F32 * net.abs())
        edl = edl + before(eww) + 12 * F32 * torch.cumsum(ww.abs(), 0) + esr
        dl = span.abs() + suffix(v).abs() + before(ww).abs() + sr.abs()
        xu = (self.G.sum(0) + self.self_[0] + w).abs()
        exu = self.eG.sum(0) + self.self_[1] + ew + 30 * F32 * (col + self.self_[0].abs() + w.abs())
        return exu, xu, edl + 8 * F32 * dl, dl


def suffix(t):
    return torch.flip(torch.cumsum(torch.flip(t, [0]), 0), [0])


def before(t):
    return torch.cumsum(t, 0) - t


def case_bounds(case, seed=1):
    B, N, H, G, D, M, dtype, lengths, decay = case
    p, dy, _ = inputs(B, N, H, G, D, M, dtype, seed, decay)
    h = place(p, H, G, D, M, "cpu")
    a = [h[k] for k in PARAMS]
    want = plain64.scan(*a, None, lengths, dy)
    b = gate_bounds(*a, lengths, dy)
    return (*a, lengths, dy), want, {n: b[n] + BF16 * (want[n].abs() + b[n]) for n in NAMES}


def fails(got, want, b, name):
    with pytest.raises(AssertionError):
        within(got, want, b, name)


def bf16_terms(n):
    def kept(t):
        left, total = t, torch.zeros_like(t)
        for _ in range(n):
            part = left.float().bfloat16().double()
            left, total = left - part, total + part
        return total
    return kept


@pytest.mark.parametrize("case", BF16_CASES)
def test_bounds_are_below_the_values(case):
    """Zeros and flipped signs are outside the bounds, and nearly every entry by itself."""
    _, want, b = case_bounds(case)
    for n in NAMES:
        at = want[n] != 0
        if case[1] == 1 and n == "dA":  # a single row from a zero state feels no decay
            assert not at.any() and float(b[n].abs().max()) == 0.0
            continue
        slow = case[8] < 1.0  # dA and ddt_bias are then small beside what they cancel from
        assert float(b[n].norm()) < (0.9 if slow and n != "ddt" else 0.05) * float(want[n].norm()), n
        fails(torch.zeros_like(want[n]), want[n], b[n], n)
        fails(-want[n], want[n], b[n], n)
        assert slow or float((b[n][at] < want[n][at].abs()).double().mean()) > 0.9, n


@pytest.mark.parametrize("case", [c for c in BF16_CASES if c[1] > 256])
def test_bounds_refuse_other_sums(case):
    """The kernels' sums in 64 bits are the recurrence's; with states of two terms they are within the bounds; with one
    row's pairs missing, or those outside the diagonal blocks, they are not."""
    args, want, b = case_bounds(case)
    same, every = (lambda t: t), (lambda t: t)
    for n, t in gate_values(args, same, every).items():
        within(t, want[n], 1e-9 * (1 + want[n].abs()), n)
    for n, t in gate_values(args, bf16_terms(2), every).items():
        within(t, want[n], b[n], n)

    def no_row(G):
        G = G.clone()
        G[min(40, len(G) - 1)] = 0
        return G

    def near(G):
        k = torch.arange(len(G)) // 32
        return torch.where(k[:, None] == k[None, :], G, 0.0)
    for kept, pairs, names in ((same, no_row, NAMES[:1] if case[8] < 1.0 else NAMES), (same, near, NAMES)):
        got = gate_values(args, kept, pairs)
        for n in names:
            fails(got[n], want[n], b[n], n)


@pytest.mark.parametrize("case", [c for c in BF16_CASES if c[1] > 256 and c[4] == 16 and c[5] < 64])
def test_bounds_refuse_states_of_one_term(case):
    args, want, b = case_bounds(case)
    fails(gate_values(args, bf16_terms(1), lambda t: t)["ddt"], want["ddt"], b["ddt"], "ddt")


@pytest.mark.gpu
@pytest.mark.parametrize("case", BF16_CASES)
def test_gate_gradients(cuda, linattn, case):
    B, N, H, G, D, M, dtype, lengths, decay = case
    args, want, b = case_bounds(case)
    d = place(inputs(B, N, H, G, D, M, dtype, 1, decay)[0], H, G, D, M, cuda)
    got = dict(zip(("dx", "ddt", "dA", "dBm", "dCm", "dskip", "ddt_bias"), linattn.scan_bwd(*[d[k] for k in PARAMS], args[-1].to(cuda), lengths=to_cuda(lengths))))
    for n in NAMES:
        within(got[n], want[n], b[n], n)


FEW = [(1, 1, 4, 1, 64, 64), (2, 1, 2, 2, 32, 64), (1, 3, 3, 1, 64, 32)]  # B, N, H, G, D, M


def few_rows(B, N, H, G, D, M):
    """The scan of a few rows from a zero state, and the final state's bound: three bf16 terms of the scaled row."""
    p, _, _ = inputs(B, N, H, G, D, M, "bf16", 12)
    h = place(p, H, G, D, M, "cpu")
    a = [h[k] for k in PARAMS]
    want, size = (plain64.scan(*a, torch.zeros(B, H, D, M), size=s)["S"] for s in (False, True))
    delta, _, A = plain64.gate(p["dt"], p["A"], p["dt_bias"], None)
    z, tot = float((p["dt"].double() + p["dt_bias"].double()).abs().max()), float((delta * A.abs()).sum(1).max())
    # decays and delta as in Chunk; a few rows lie in one step of the products; the accumulators, the carry
    return p, a, want, ((9 + z + 16 + 12) * tot + 24 + 8 + z + 11 + 8) * F32 * size + 2.0 ** -24 * size


@pytest.mark.parametrize("B,N,H,G,D,M", FEW[:2])
def test_bounds_refuse_two_terms_of_the_state(B, N, H, G, D, M):
    _, (x, dt, A, Bm, Cm, skip, bias), want, b = few_rows(B, N, H, G, D, M)
    delta, _, A = plain64.gate(dt, A, bias, None)
    cum = torch.cumsum(delta * A, 1)
    u = (delta * torch.exp(cum[:, -1:] - cum))[..., None] * x.double()
    for n, f in ((3, within), (2, fails)):
        f(torch.einsum("bnhd,bnhm->bhdm", Bm.double().repeat_interleave(H // G, 2), bf16_terms(n)(u)), want, b, "S")


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,H,G,D,M", FEW)
def test_final_state_of_few_rows(cuda, linattn, B, N, H, G, D, M):
    p, _, want, b = few_rows(B, N, H, G, D, M)
    d, S = place(p, H, G, D, M, cuda), torch.zeros(B, H, D, M, device=cuda)
    linattn.scan_fwd(*[d[k] for k in PARAMS], S=S)
    within(S, want, b, "S")


def one_live_row(N, row, heavy):
    """Rows that forget everything (`heavy`) before rows that hardly do; x is not zero in one of the latter alone."""
    g = torch.Generator().manual_seed(13)
    B, H, G, D, M = 2, 3, 1, 32, 64
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, Bm, Cm = torch.zeros(B, N, H, M), r(B, N, G, D).bfloat16(), r(B, N, G, D).bfloat16()
    x[:, row] = r(B, H, M)
    dt = torch.where(torch.arange(N)[None, :, None] < heavy, 1.0, -5.0) + 0.25 * r(B, N, H)
    a = [x.bfloat16(), dt.bfloat16(), torch.tensor([-16.0, -11.0, -13.5]).bfloat16(), Bm, Cm, None, None]
    want, size = (plain64.scan(*a, torch.zeros(B, H, D, M), size=s)["S"] for s in (False, True))
    delta, _, A = plain64.gate(*a[1:3], None, None)
    z, tot = float(dt.abs().max()) + 1, float((delta * A.abs())[:, row + 1:].sum(1).max())
    return a, (delta, A), want, ((9 + z + 16 + 12) * tot + 24 + 8 + z + 11 + 8 + 4 * (N // CH + 1)) * F32 * size + 2.0 ** -24 * size


ROWS = [(128, 126, 120), (128, 61, 60), (224, 215, 212)]


@pytest.mark.parametrize("N,row,heavy", ROWS)
def test_bounds_refuse_a_difference_of_sums(N, row, heavy):
    """The decay from a row to the end of its 32-row block in fp32: as a sum of its own, and as a difference of two."""
    (x, _, _, Bm, _, _, _), (delta, A), want, b = one_live_row(N, row, heavy)
    l, first = (delta * A).float(), row // 32 * 32
    block = l[:, first:first + 32]
    wp = torch.cumsum(block, 1)
    rest = (delta * A)[:, first + 32:].sum(1)
    for f, near in ((within, block[:, row - first + 1:].flip(1).sum(1)), (fails, wp[:, -1] - wp[:, row - first])):
        w = delta[:, row] * torch.exp(near.double() + rest)
        f(torch.einsum("bd,bhm->bhdm", Bm[:, row, 0].double(), w[..., None] * x[:, row].double()), want, b, "S")


@pytest.mark.gpu
@pytest.mark.parametrize("N,row,heavy", ROWS)
def test_state_behind_rows_that_forget(cuda, linattn, N, row, heavy):
    a, _, want, b = one_live_row(N, row, heavy)
    S = torch.zeros(want.shape, device=cuda)
    linattn.scan_fwd(*[None if t is None else t.to(cuda) for t in a], S=S)
    within(S, want, b, "S")
