"""The layer norm against 64 bits, within bounds of the roundings of fp32 (around64)."""
import pytest
import torch

import around64
from around64 import rounded
from plain64 import within

T = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(B, N, C, dtype, pad=0, seed=0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = T[dtype]
    return (r(B, N, C + pad) + shift).to(t), r(C).to(t), r(C).to(t), r(B, N, C + 2 * pad).to(t), r(B, N, C).to(t), r(B, N, C).to(t)


CASES = [  # B, N, C, groups, dtype, pad, lengths
    (1, 1, 2, 1, "f32", 0, None),
    (1, 3, 8, 1, "bf16", 0, None),
    (2, 5, 33, 1, "f32", 0, [5, 2]),
    (3, 17, 64, 1, "bf16", 8, [17, 0, 4]),      # an empty sequence
    (2, 9, 64, 1, "bf16", 3, None),             # rows off the vectors
    (2, 40, 320, 5, "bf16", 0, [40, 33]),       # heads of 64, a number of them that no block holds whole
    (2, 40, 96, 3, "f32", 4, None),
    (1, 60, 70, 7, "f32", 0, None),             # heads of ten columns
    (2, 11, 256, 1, "f32", 0, None),
    (2, 11, 512, 1, "bf16", 0, None),
    (2, 11, 777, 1, "f32", 0, [11, 7]),
    (2, 11, 1000, 1, "bf16", 0, None),
    (2, 6, 2048, 1, "bf16", 0, None),
    (2, 6, 2047, 1, "bf16", 0, None),
    (2, 6, 2052, 1, "f32", 0, None),
    (1, 5, 4104, 1, "bf16", 8, None),
    (1, 5, 4100, 1, "f32", 0, None),
    (1, 3, 8192, 1, "bf16", 0, None),
    (1, 3, 8192, 1, "f32", 0, None),
    (1, 3, 8191, 1, "bf16", 0, None),
    (1, 700, 64, 1, "bf16", 0, None),           # many rows a block
    (1, 5000, 40, 4, "f32", 0, None),
    (1, 9, 65, 65, "f32", 0, None),             # one column a group: y = b
]


@pytest.mark.gpu
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("B,N,C,G,dtype,pad,lengths", CASES)
def test_forward_and_gradients(cuda, linattn, B, N, C, G, dtype, pad, lengths, residual):
    x, w, b, res, dy, ds = inputs(B, N, C, dtype, pad, C)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=cuda)
    res, ds = (res[..., :C], ds) if residual else (None, None)
    dev = lambda t: None if t is None else t.to(cuda)  # noqa: E731
    xd, rd = dev(x)[..., :C], None if res is None else dev(inputs(B, N, C, dtype, pad, C)[3])[..., :C]
    y, s, mean, rstd = linattn.norm_fwd(xd, dev(w), dev(b), residual=rd, groups=G, lengths=n)
    want = around64.norm(x[..., :C], w, b, res, G, 1e-5, lengths, dy, ds)
    live = torch.arange(N)[None, :] < torch.tensor([N] * B if lengths is None else lengths)[:, None]
    got = {"y": y, "mean": mean, "rstd": rstd}
    if residual:
        got["s"] = s
    else:
        assert s is xd
    got["dx"], got["dw"], got["db"] = linattn.norm_bwd(s, dev(w), mean, rstd, dev(dy), dev(ds), groups=G, lengths=n)
    for name, t in got.items():
        fine = name in ("mean", "rstd")
        within(t, want[name][0], want[name][1] if fine else rounded(*want[name], dtype) * (name != "s"), name)
    y2 = linattn.norm_fwd(xd, dev(w), None, residual=rd, groups=G, eps=0.5, lengths=n)[0]
    want = around64.norm(x[..., :C], w, None, res, G, 0.5, lengths)["y"]
    within(y2, want[0], rounded(*want, dtype), "y without a bias")
    dx, dw, db = linattn.norm_bwd(s, dev(w), mean, rstd, dev(dy), dev(ds), groups=G, bias=False, lengths=n)
    assert db is None and torch.equal(dx, got["dx"]) and torch.equal(dw, got["dw"])
    assert live.shape == (B, N)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(7, 48), (1, 64), (300, 33)])
def test_rows_of_a_matrix(cuda, linattn, shape):
    """[N, C]: the same as [1, N, C]."""
    x, w, b, res, dy, ds = inputs(1, *shape, "bf16", 0, 3)
    a = [t.to(cuda) for t in (x, w, b, res)]
    y, s, mean, rstd = linattn.norm_fwd(*a)
    y2, s2, mean2, rstd2 = linattn.norm_fwd(a[0][0], a[1], a[2], a[3][0])
    assert torch.equal(y[0], y2) and torch.equal(s[0], s2) and torch.equal(mean[0], mean2)
    g = linattn.norm_bwd(s, a[1], mean, rstd, dy.to(cuda))
    g2 = linattn.norm_bwd(s2, a[1], mean2, rstd2, dy[0].to(cuda))
    assert torch.equal(g[0][0], g2[0]) and torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_far_from_zero_and_constant_rows(cuda, linattn, dtype):
    """Means of a thousand deviations, and rows without any: the variance is of differences, never negative."""
    x, w, b, _, dy, _ = inputs(2, 30, 192, dtype, 0, 4, shift=1000.0)
    x[0, 3], x[1, 7] = 5.0, 0.0
    y, s, mean, rstd = linattn.norm_fwd(x.to(cuda), w.to(cuda), b.to(cuda))
    got = linattn.norm_bwd(s, w.to(cuda), mean, rstd, dy.to(cuda))
    want = around64.norm(x, w, b, dy=dy)
    for name, t in zip(("y", "mean", "rstd", "dx", "dw", "db"), (y, mean, rstd, *got)):
        within(t, want[name][0], want[name][1] if name in ("mean", "rstd") else rounded(*want[name], dtype), name)


@pytest.mark.gpu
def test_padded_rows_are_not_read(cuda, linattn):
    x, w, b, res, dy, ds = (t.to(cuda) for t in inputs(3, 50, 64, "bf16", 0, 5))
    n = torch.tensor([0, 21, 50], dtype=torch.int32, device=cuda)

    def run():
        y, s, mean, rstd = linattn.norm_fwd(x, w, b, residual=res, groups=2, lengths=n)
        return [y, s, mean, rstd, *linattn.norm_bwd(s, w, mean, rstd, dy, ds, groups=2, lengths=n)]

    clean = run()
    for t in (x, res, dy, ds):
        t[0], t[1, 21:] = float("nan"), float("inf")
    for a, c in zip(clean, run()):
        assert torch.equal(a, c)
    for t in clean[:5]:
        assert float(t[0].abs().max()) == 0.0 and float(t[1, 21:].abs().max()) == 0.0


@pytest.mark.gpu
def test_live_nan(cuda, linattn):
    """A NaN stays in its group of its row."""
    x, w, b, *_ = (t.to(cuda) for t in inputs(2, 9, 96, "f32", 0, 6))
    clean = linattn.norm_fwd(x, w, b, groups=3)[0]
    x[1, 4, 40] = float("nan")
    y = linattn.norm_fwd(x, w, b, groups=3)[0]
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1, 4, 32:64] = True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], clean[~bad])


@pytest.mark.gpu
def test_autograd(cuda, linattn):
    """Gradients through y, through s and through both; a sum that nothing else reads."""
    x, w, b, res, dy, ds = (t.to(cuda) for t in inputs(2, 13, 48, "bf16", 0, 7))
    leaves = [t.requires_grad_(True) for t in (x, w, b, res)]
    y, s = linattn.layer_norm(x, w, b, res, groups=3)
    with torch.no_grad():
        yf, sf, mean, rstd = linattn.norm_fwd(x, w, b, res, groups=3)
    assert torch.equal(y, yf) and torch.equal(s, sf)
    for gy, gs in ((dy, ds), (dy, None), (None, ds)):
        want = linattn.norm_bwd(sf, w.detach(), mean, rstd, torch.zeros_like(dy) if gy is None else gy, gs, groups=3)
        outs, grads = zip(*[(o, g) for o, g in ((y, gy), (s, gs)) if g is not None])
        got = torch.autograd.grad(outs, leaves, grads, retain_graph=True)
        for a, c in zip(got, (want[0], want[1], want[2], want[0])):
            assert torch.equal(a, c)
    y = linattn.layer_norm(x, w)
    got = torch.autograd.grad(y, [x, w], dy)
    with torch.no_grad():
        _, sf, mean, rstd = linattn.norm_fwd(x, w)
    want = linattn.norm_bwd(sf, w.detach(), mean, rstd, dy, bias=False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_gradients_against_differences(cuda, linattn):
    x, w, b, _, dy, _ = inputs(2, 5, 24, "f32", 0, 8)
    leaves = [t.to(cuda).requires_grad_(True) for t in (x, w, b)]
    grads = torch.autograd.grad(linattn.layer_norm(*leaves, groups=2), leaves, dy.to(cuda))
    g = torch.Generator().manual_seed(9)

    def form(x, w, b):
        v = x.unflatten(-1, (2, 12))
        v = v - v.mean(-1, keepdim=True)
        return (v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5)).flatten(2) * w + b

    host = [x.double(), w.double(), b.double()]
    for j, d in enumerate(grads):
        v = torch.randn(d.shape, generator=g).double()
        at = lambda e: float((form(*[t + e * v if k == j else t for k, t in enumerate(host)]) * dy.double()).sum())  # noqa: E731
        fd = (at(1e-5) - at(-1e-5)) / 2e-5
        size = float((d.double().cpu().abs() * v.abs()).sum())
        assert abs(fd - float((d.double().cpu() * v).sum())) <= 2e-5 * size


@pytest.mark.gpu
def test_offsets_beyond_32_bits(cuda, linattn):
    C = 2048
    N = (1 << 31) // C + 500
    x = torch.empty(N, C, dtype=torch.bfloat16, device=cuda).normal_()
    w, b = torch.randn(C, device=cuda).bfloat16(), torch.randn(C, device=cuda).bfloat16()
    y, s, mean, rstd = linattn.norm_fwd(x, w, b)
    part = linattn.norm_fwd(x[-300:], w, b)
    assert torch.equal(y[-300:], part[0]) and torch.equal(mean[-300:], part[2])
    dx = linattn.norm_bwd(s, w, mean, rstd, x)[0]
    assert torch.equal(dx[-300:], linattn.norm_bwd(x[-300:], w, part[2], part[3], x[-300:])[0])


FAKE = 1 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(y=FAKE + 8), 1), (dict(x=FAKE + 2), 1), (dict(w=FAKE + 4), 1), (dict(b=FAKE + 4), 1),
    (dict(res=FAKE), 1), (dict(res=FAKE + 1, s=FAKE), 1), (dict(mean=None), 1), (dict(rstd=FAKE + 8), 1), (dict(lengths=FAKE + 2), 1), (dict(B=0), 1),
    (dict(N=0), 1), (dict(C=0), 1), (dict(G=0), 1), (dict(G=3), 1), (dict(C=65540, ldx=65540), 1), (dict(ldx=7), 1), (dict(res=FAKE, s=FAKE, ldr=7), 1),
    (dict(C=8200, ldx=8200), 2), (dict(B=1 << 16, N=1 << 16), 1), (dict(B=1 << 14, N=1 << 14, G=8), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(dt=2), 1),
])
def test_refusals(linattn, kw, code):
    a = dict(x=FAKE, res=None, w=FAKE, b=None, lengths=None, y=FAKE, s=None, mean=FAKE, rstd=FAKE, eps=1e-5, B=1, N=4, C=8, G=1, ldx=8, ldr=8, dt=0)
    a.update(kw)
    assert linattn.lib().la_norm_fwd(*[a[n] for n in ("x", "res", "w", "b", "lengths", "y", "s", "mean", "rstd", "eps", "B", "N", "C", "G", "ldx", "ldr", "dt")],
                                     None) == code


def test_refusals_of_the_gradients(linattn):
    L, F = linattn.lib(), FAKE
    need = linattn.la_norm_workspace_bytes(1, 4, 8, 1, 0)
    assert need > 0 and linattn.la_norm_workspace_bytes(1, 4, 8, 3, 0) == 0
    bwd = lambda mean, ds, db, ws, wsb: L.la_norm_bwd(F, F, mean, F, None, F, ds, F, F, db, ws, wsb, 1, 4, 8, 1, 8, 0, None)  # noqa: E731
    assert bwd(None, None, None, F, need) == linattn.LA_ERR_INVALID_ARG
    assert bwd(F, F + 4, None, F, need) == linattn.LA_ERR_INVALID_ARG
    assert bwd(F, None, F + 8, F, need) == linattn.LA_ERR_INVALID_ARG
    assert bwd(F, None, None, None, 0) == linattn.LA_ERR_WORKSPACE
    assert bwd(F, None, None, F, need - 1) == linattn.LA_ERR_WORKSPACE


def test_binding_refuses(linattn):
    x, w = torch.zeros(2, 5, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA device"):
        linattn.norm_fwd(x, w)
    with pytest.raises(ValueError, match="w: shape"):
        linattn.norm_fwd(x, torch.zeros(9))
    with pytest.raises(TypeError, match="b: "):
        linattn.norm_fwd(x, w, w.bfloat16())
    with pytest.raises(ValueError, match="residual: shape"):
        linattn.norm_fwd(x, w, None, x[:, :4])
    with pytest.raises(ValueError, match="does not divide"):
        linattn.norm_fwd(x, w, groups=3)
    with pytest.raises(ValueError, match="lengths"):
        linattn.norm_fwd(x[0], w, lengths=torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError, match="dense"):
        linattn.norm_fwd(torch.zeros(2, 8, 5).transpose(1, 2), w)
    with pytest.raises(ValueError, match="mean: shape"):
        linattn.norm_bwd(x, w, torch.zeros(2, 5), torch.zeros(2, 5), x)
