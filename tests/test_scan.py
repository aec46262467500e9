"""The selective scan against a row-by-row 64-bit recurrence.

Bounds, element by element: every output is a sum of products whose absolute
values sum to its size (``plain64.scan(size=True)``).  In fp32 a sum over a chunk
and the carried states rounds by less than 3 x 64 half steps of that size and the
decays add ``scan_step_size``; the carry over c chunks adds 2 roundings a chunk.
With bf16 inputs the scores and the carried states are rounded to bf16 once
before their products (half a step each; a term passes through one of the two)
and the result once more.  (Of the gradients the gate's, and of the states the last one, are
rounded less: test_scan_bounds.py has the bounds of just that.)
"""
import pytest
import torch

import plain64
from plain64 import BF16, F32, within

T = {"f32": torch.float32, "bf16": torch.bfloat16}
PARAMS = ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias")


def inputs(B, N, H, G, D, M, dtype, seed=0, decay=1.0):
    """x, Bm and Cm as slices of one row buffer, and dy, S."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = T[dtype]
    rows = r(B, N, H * M + 2 * G * D + 16).to(t)
    p = {"rows": rows, "dt": (0.5 * r(B, N, H)).to(t), "A": (-decay * (1 + 7 * torch.rand(H, generator=g))).to(t),
         "skip": r(H).to(t), "dt_bias": (-3 + r(H)).to(t)}
    return p, r(B, N, H, M).to(t), r(B, H, D, M)


def place(p, H, G, D, M, device):
    rows = p["rows"].to(device)
    q = {k: v.to(device) for k, v in p.items() if k != "rows"}
    q["x"] = rows[..., :H * M].unflatten(-1, (H, M))
    q["Bm"] = rows[..., H * M:H * M + G * D].unflatten(-1, (G, D))
    q["Cm"] = rows[..., H * M + G * D:H * M + 2 * G * D].unflatten(-1, (G, D))
    return q


def rel(p, N, dtype, out_rounding=True):
    """The relative bound on an output's size."""
    c = plain64.scan_step_size(p["dt"], p["A"], p["dt_bias"], 64 if dtype == "f32" else 128)
    e = 3 * 64 * F32 + 2 * c + 2 * (N // 64 + 1) * F32
    if dtype == "bf16":
        e += (1 + BF16) * BF16 * (2 if out_rounding else 1)
    return e


CASES = [  # B, N, H, G, D, M, dtype, lengths
    (1, 1, 1, 1, 16, 16, "f32", None),
    (1, 1, 1, 1, 64, 64, "bf16", None),
    (2, 5, 2, 1, 32, 16, "f32", [5, 0]),
    (1, 64, 2, 2, 16, 64, "f32", None),
    (1, 65, 2, 1, 64, 32, "f32", None),
    (2, 200, 4, 2, 64, 64, "f32", [129, 200]),
    (1, 130, 3, 3, 32, 32, "bf16", None),
    (2, 257, 4, 1, 64, 64, "bf16", [257, 128]),
    (3, 300, 2, 2, 16, 64, "bf16", [0, 1, 300]),
    (1, 500, 6, 2, 64, 16, "bf16", None),
    (1, 140, 12, 1, 64, 32, "bf16", [139]),
    (2, 129, 5, 5, 32, 64, "bf16", None),
]


def to_cuda(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,H,G,D,M,dtype,lengths", CASES)
def test_forward(cuda, linattn, B, N, H, G, D, M, dtype, lengths):
    p, _, S = inputs(B, N, H, G, D, M, dtype)
    h, d = place(p, H, G, D, M, "cpu"), place(p, H, G, D, M, cuda)
    n = to_cuda(lengths)
    for S0, skip, bias in ((None, True, True), (S, True, True), (S, False, False)):
        a = [h[k] if k not in ("skip", "dt_bias") or (skip if k == "skip" else bias) else None for k in PARAMS]
        want = plain64.scan(*a, S0, lengths)
        size = plain64.scan(*a, S0, lengths, size=True)
        q = dict(p) if bias else dict(p, dt_bias=None)
        Sd = None if S0 is None else S0.to(cuda)
        ad = [d[k] if k not in ("skip", "dt_bias") or (skip if k == "skip" else bias) else None for k in PARAMS]
        y = linattn.scan_fwd(*ad, S=Sd, lengths=n)
        within(y, want["y"], rel(q, N, dtype) * size["y"], "y")
        if S0 is not None:
            # the state is fp32-accurate for either type: bf16 operands are split into two terms (2^-16)
            e = rel(q, N, "f32") + (2.0 ** -16 if dtype == "bf16" else 0)
            within(Sd, want["S"], e * size["S"], "S")


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,H,G,D,M,dtype,lengths", CASES)
def test_backward(cuda, linattn, B, N, H, G, D, M, dtype, lengths):
    p, dy, _ = inputs(B, N, H, G, D, M, dtype, 1)
    h, d = place(p, H, G, D, M, "cpu"), place(p, H, G, D, M, cuda)
    a = [h[k] for k in PARAMS]
    want = plain64.scan(*a, None, lengths, dy)
    size = plain64.scan(*a, None, lengths, dy, size=True)
    got = linattn.scan_bwd(*[d[k] for k in PARAMS], dy.to(cuda), lengths=to_cuda(lengths))
    for k, g in zip(PARAMS, got):
        # ddt and the parameters pass two roundings before the last one: the scores of dx and the carried states
        e = rel(p, N, dtype) + (BF16 if dtype == "bf16" and k in ("dt", "A", "dt_bias") else 0)
        within(g, want["d" + k], e * size["d" + k], "d" + k)


@pytest.mark.gpu
@pytest.mark.parametrize("N,H,G,D,M,dtype,lengths", [
    (4300, 1, 1, 16, 16, "f32", [4290]),      # 68 chunks: the carry in segments
    (8800, 2, 1, 16, 32, "bf16", [8500]),     # 69
    (300, 40, 1, 16, 16, "bf16", None),       # more heads to a group than a block takes
])
def test_long_and_wide(cuda, linattn, N, H, G, D, M, dtype, lengths):
    test_forward(cuda, linattn, 1, N, H, G, D, M, dtype, lengths)
    test_backward(cuda, linattn, 1, N, H, G, D, M, dtype, lengths)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_offsets_beyond_32_bits(cuda, linattn, dtype):
    """More than 2^31 elements; the last rows against the recurrence over them alone, which a decay of
    at least exp(-1) a row makes exact after 200 rows."""
    H, G, D, M, tail, warm = 64, 1, 16, 32, 400, 200
    N = (1 << 31) // (H * M) + 777
    t, rows = T[dtype], torch.empty(1, N, H * M, dtype=T[dtype], device=cuda).normal_()
    bc = torch.empty(1, N, 2 * G * D, dtype=t, device=cuda).normal_()
    dt = torch.full((1, N, H), 1.0, dtype=t, device=cuda)
    A, skip = torch.full((H,), -1.0, dtype=t, device=cuda), torch.ones(H, dtype=t, device=cuda)
    x, b, c = rows.unflatten(-1, (H, M)), bc[..., :G * D].unflatten(-1, (G, D)), bc[..., G * D:].unflatten(-1, (G, D))
    args = [x, dt, A, b, c, skip, None]
    cpu = [a if a is None else (a[:, -tail:] if a.dim() > 1 else a).cpu() for a in args]
    p = {"dt": cpu[1], "A": cpu[2], "dt_bias": None}
    y = linattn.scan_fwd(*args)[:, -tail:].cpu()
    want, size = plain64.scan(*cpu, None), plain64.scan(*cpu, None, size=True)
    within(y[:, warm:], want["y"][:, warm:], rel(p, tail, dtype) * size["y"][:, warm:], "y")
    dy = torch.zeros_like(x)
    dy[:, -tail + warm:] = torch.empty_like(dy[:, -tail + warm:]).normal_()
    g = dy[:, -tail:].cpu()
    want, size = plain64.scan(*cpu, None, None, g), plain64.scan(*cpu, None, None, g, size=True)
    dx, ddt, dA, dB, dC, dskip, _ = linattn.scan_bwd(*args[:6], None, dy)
    for k, got in (("dx", dx), ("dBm", dB), ("dCm", dC)):
        got = got[:, -tail:].cpu()
        within(got[:, warm:], want[k][:, warm:], rel(p, tail, dtype) * size[k][:, warm:], k)
    assert float(dx[:, :1000].abs().max()) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, 1e-4, 40.0])
def test_slow_and_fast_decays(cuda, linattn, dtype, decay):
    """No decay at all, almost none, and one that forgets within a row."""
    B, N, H, G, D, M = 1, 290, 2, 1, 32, 32
    p, dy, S = inputs(B, N, H, G, D, M, dtype, 4, decay)
    p["dt_bias"] = torch.zeros_like(p["dt_bias"])
    h, d = place(p, H, G, D, M, "cpu"), place(p, H, G, D, M, cuda)
    a = [h[k] for k in PARAMS]
    want, size = plain64.scan(*a, S), plain64.scan(*a, S, size=True)
    Sd = S.to(cuda)
    y = linattn.scan_fwd(*[d[k] for k in PARAMS], S=Sd)
    within(y, want["y"], rel(p, N, dtype) * size["y"], "y")
    want, size = plain64.scan(*a, dy=dy), plain64.scan(*a, dy=dy, size=True)
    got = linattn.scan_bwd(*[d[k] for k in PARAMS], dy.to(cuda))
    for k, g in zip(PARAMS, got):
        e = rel(p, N, dtype) + (BF16 if dtype == "bf16" and k in ("dt", "A", "dt_bias") else 0)
        within(g, want["d" + k], e * size["d" + k], "d" + k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_growing_states(cuda, linattn, dtype):
    """A > 0: nothing in the chunk form needs the decays to be below one."""
    test_slow_and_fast_decays(cuda, linattn, dtype, -0.01)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,G,D,M,dtype", [(1, 1, 1, 16, 16, "f32"), (3, 4, 2, 64, 64, "bf16"), (40, 6, 1, 32, 64, "bf16"), (2, 5, 5, 64, 16, "f32")])
def test_steps_continue_a_prompt(cuda, linattn, B, H, G, D, M, dtype):
    N, cut = 140, 131
    p, _, S = inputs(B, N, H, G, D, M, dtype, 2)
    h, d = place(p, H, G, D, M, "cpu"), place(p, H, G, D, M, cuda)
    want = plain64.scan(*[h[k] for k in PARAMS], S)
    size = plain64.scan(*[h[k] for k in PARAMS], S, size=True)
    Sd = S.to(cuda)
    first = lambda t: t[:, :cut].contiguous() if t.dim() > 1 else t  # noqa: E731
    ys = [linattn.scan_fwd(*[first(d[k]) for k in PARAMS], S=Sd)]
    for t in range(cut, N):
        ys.append(linattn.scan_step(*[d[k][:, t] if d[k].dim() > 1 else d[k] for k in PARAMS], Sd)[:, None])
    within(torch.cat(ys, 1), want["y"], rel(p, N, dtype) * size["y"], "y")
    within(Sd, want["S"], (rel(p, N, "f32") + (2.0 ** -16 if dtype == "bf16" else 0)) * size["S"], "S")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padded_rows_are_not_read(cuda, linattn, dtype):
    B, N, H, G, D, M = 3, 270, 2, 1, 32, 64
    p, dy, S = inputs(B, N, H, G, D, M, dtype, 3)
    n = to_cuda([0, 200, 270])
    run = lambda d, g, S: [linattn.scan_fwd(*[d[k] for k in PARAMS], S=S, lengths=n), S, *linattn.scan_bwd(*[d[k] for k in PARAMS], g, lengths=n)]  # noqa: E731
    d = place(p, H, G, D, M, cuda)
    clean = run(d, dy.to(cuda), S.to(cuda))
    bad = dict(p, rows=p["rows"].clone(), dt=p["dt"].clone())
    gd = dy.clone()
    for b, m in ((0, 0), (1, 200)):
        bad["rows"][b, m:], bad["dt"][b, m:], gd[b, m:] = float("nan"), float("inf"), float("nan")
    dirty = run(place(bad, H, G, D, M, cuda), gd.to(cuda), S.to(cuda))
    for a, c in zip(clean, dirty):
        assert torch.equal(a, c)
    assert torch.equal(dirty[1][0].cpu(), S[0])  # an empty sequence leaves its state
    assert float(dirty[0][1, 200:].abs().max()) == 0.0


@pytest.mark.gpu
def test_gradients_against_differences(cuda, linattn):
    B, N, H, G, D, M = 1, 70, 2, 1, 16, 16
    p, dy, _ = inputs(B, N, H, G, D, M, "f32", 5)
    h, d = place(p, H, G, D, M, "cpu"), place(p, H, G, D, M, cuda)
    leaves = [d[k].contiguous().requires_grad_(True) for k in PARAMS]
    grads = torch.autograd.grad(linattn.selective_scan(*leaves), leaves, dy.to(cuda))
    g = torch.Generator().manual_seed(9)
    a = [h[k].double() for k in PARAMS]
    size = plain64.scan(*a, dy=dy, size=True)
    for i, k in enumerate(PARAMS):
        v = torch.randn(a[i].shape, generator=g).double()
        at = lambda e: float((plain64.scan(*[t + e * v if j == i else t for j, t in enumerate(a)])["y"] * dy.double()).sum())  # noqa: E731
        fd = (at(1e-5) - at(-1e-5)) / 2e-5
        bound = float((size["d" + k] * v.abs()).sum()) * rel(p, N, "f32") + 1e-6 * abs(fd)  # differences: ~h^2 of third derivatives
        assert abs(fd - float((grads[i].double().cpu() * v).sum())) <= bound, k


@pytest.mark.gpu
def test_other_stream_and_unwritten_guards(cuda, linattn):
    """On a side stream, into buffers with guard rows around them, from poisoned outputs and workspace."""
    la = linattn
    B, N, H, G, D, M = 2, 150, 4, 2, 64, 64
    p, dy, S = inputs(B, N, H, G, D, M, "bf16", 6)
    d = place(p, H, G, D, M, cuda)
    ref = la.scan_fwd(*[d[k] for k in PARAMS], S=S.to(cuda))
    grads = la.scan_bwd(*[d[k] for k in PARAMS], dy.to(cuda))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        buf = torch.full((B * N * H * M + 64,), 7.0, dtype=torch.bfloat16, device=cuda)
        ws = torch.full((la.la_scan_workspace_bytes(0, B, H, G, N, D, M, la.LA_BF16),), 255, dtype=torch.uint8, device=cuda)
        y, Sd, ld = buf[32:-32].view(B, N, H, M), S.to(cuda), d["x"].stride(1)
        la.la_scan_fwd(*[d[k] for k in PARAMS], None, Sd, y, ws, B, H, G, N, D, M, ld, H, ld, ld, la.LA_BF16)
        ws = torch.full((la.la_scan_workspace_bytes(1, B, H, G, N, D, M, la.LA_BF16),), 255, dtype=torch.uint8, device=cuda)
        outs = [torch.full_like(t, float("nan")) for t in grads]
        la.la_scan_bwd(*[d[k] for k in PARAMS], None, dy.to(cuda), *[outs[i] for i in (0, 1, 2, 3, 4, 5, 6)], ws, B, H, G, N, D, M, ld, H, ld, ld, la.LA_BF16)
    s.synchronize()
    assert torch.equal(y, ref) and (buf[:32] == 7).all() and (buf[-32:] == 7).all()
    for a, b in zip(outs, grads):
        assert torch.equal(a, b)
    la.check_device_status()


FAKE = 1 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(dt=None), 1), (dict(A=None), 1), (dict(Bm=FAKE + 8), 1), (dict(Cm=None), 1), (dict(dt=FAKE + 2), 1),
    (dict(skip=FAKE + 4), 1), (dict(dt_bias=FAKE + 4), 1), (dict(S=FAKE + 4), 1), (dict(y=None), 1), (dict(lengths=FAKE + 1), 1),
    (dict(G=3), 1), (dict(G=0), 1), (dict(H=32768, ldx=1 << 20, lddt=32768), 1), (dict(H=0), 1), (dict(N=0), 1), (dict(B=65536), 1), (dict(D=128), 2), (dict(M=24), 2), (dict(D=0), 1),
    (dict(ldx=60), 1), (dict(ldx=66), 1), (dict(ldb=15), 1), (dict(ldc=18), 1), (dict(lddt=3), 1), (dict(t=9), 1),
    (dict(wsb=16), 5), (dict(ws=None), 5), (dict(ws=FAKE + 4), 1),
])
def test_refusals(linattn, kw, code):
    a = dict(x=FAKE, dt=FAKE, A=FAKE, Bm=FAKE, Cm=FAKE, skip=None, dt_bias=None, lengths=None, S=FAKE, y=FAKE, ws=FAKE, wsb=1 << 40,
             B=1, H=4, G=1, N=300, D=16, M=16, ldx=64, lddt=4, ldb=16, ldc=16, t=0)
    a.update(kw)
    L = linattn.lib()
    order = ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias", "lengths", "S", "y", "ws", "wsb", "B", "H", "G", "N", "D", "M", "ldx", "lddt", "ldb", "ldc", "t")
    assert L.la_scan_fwd(*[a[k] for k in order], None) == code


def test_refusals_of_the_other_calls(linattn):
    L, F = linattn.lib(), FAKE
    size = (1, 4, 1, 300, 16, 16, 64, 4, 16, 16, 0)
    bwd = lambda skip, dskip, ws, wsb: L.la_scan_bwd(F, F, F, F, F, skip, None, None, F, F, F, F, F, F, dskip, None, ws, wsb, *size, None)  # noqa: E731
    need = linattn.la_scan_workspace_bytes(1, 1, 4, 1, 300, 16, 16, 0)
    assert need > linattn.la_scan_workspace_bytes(0, 1, 4, 1, 300, 16, 16, 0) > 0
    assert linattn.la_scan_workspace_bytes(1, 1, 4, 3, 300, 16, 16, 0) == 0
    assert bwd(None, None, F, need - 1) == linattn.LA_ERR_WORKSPACE
    assert bwd(F, None, F, need) == linattn.LA_ERR_INVALID_ARG
    step = lambda S, B=1, ldx=64: L.la_scan_step(F, F, F, F, F, None, None, S, F, B, 4, 1, 16, 16, ldx, 4, 16, 16, 0, None)  # noqa: E731
    assert step(None) == 1 and step(F, B=(1 << 18) + 1) == 1 and step(F, ldx=63) == 1


def test_binding_refuses_strides_and_sizes_beyond_the_interface(linattn):
    far = lambda *s: torch.empty_strided(s, (1 << 33, 1 << 32, 16, 1)[-len(s):], device="meta")  # noqa: E731
    x, dt, A, b = (torch.empty(*s, device="meta") for s in ((2, 1, 4, 16), (2, 1, 4), (4,), (2, 1, 1, 16)))
    with pytest.raises(ValueError, match="apart, at most"):
        linattn.scan_fwd(far(2, 1, 4, 16), dt, A, b, b)
    with pytest.raises(ValueError, match="apart, at most"):
        linattn.scan_step(far(2, 4, 16).as_strided((2, 4, 16), (1 << 32, 16, 1)), dt[:, 0], A, b[:, 0], b[:, 0], None, None, b)
    with pytest.raises(ValueError, match="sizes above"):
        linattn.scan_fwd(torch.empty(1, (1 << 32) + 5, 4, 16, device="meta"), dt, A, b, b)


@pytest.mark.gpu
def test_no_second_derivatives(cuda, linattn):
    x, b = torch.randn(1, 3, 2, 16, device=cuda, requires_grad=True), torch.randn(1, 3, 1, 16, device=cuda)
    y = linattn.selective_scan(x, b[..., 0, :2].contiguous(), -torch.ones(2, device=cuda), b, b)
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_binding_refuses(linattn):
    z = torch.zeros
    x, dt, A, b = z(2, 5, 4, 16), z(2, 5, 4), z(4), z(2, 5, 1, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        linattn.scan_fwd(x, dt, A, b, b)
    with pytest.raises(ValueError, match="dt: shape"):
        linattn.scan_fwd(x, dt[:, :4], A, b, b)
    with pytest.raises(TypeError, match="A:"):
        linattn.scan_fwd(x, dt, A.bfloat16(), b, b)
    with pytest.raises(ValueError, match="Cm: shape"):
        linattn.scan_fwd(x, dt, A, b, z(2, 5, 2, 16))
    with pytest.raises(ValueError, match="dense"):
        linattn.scan_fwd(z(2, 5, 16, 4).transpose(2, 3), dt, A, b, b)
    with pytest.raises(ValueError, match="S: shape"):
        linattn.scan_fwd(x, dt, A, b, b, S=z(2, 4, 16, 17))


@pytest.mark.gpu
@pytest.mark.parametrize("N,dtype", [(64 * 65, "f32"), (64 * 66, "f32"), (128 * 66 - 5, "bf16"), (128 * 79, "bf16")])
def test_segments_of_the_carry_start_from_the_given_state(cuda, linattn, N, dtype):
    """Above 64 chunks the carry runs in segments, all of which start from S while the last one replaces it (at
    66 chunks that one is a single chunk and ends first).  With hardly any decay S reaches every row of y."""
    B, H, G, D, M = 2, 3, 1, 16, 16
    p, _, S = inputs(B, N, H, G, D, M, dtype, 7, 1e-4)
    S = 8 * S
    h, d = place(p, H, G, D, M, "cpu"), place(p, H, G, D, M, cuda)
    want, size = (plain64.scan(*[h[k] for k in PARAMS], S, size=s) for s in (False, True))
    runs = []
    for _ in range(6):
        Sd = S.to(cuda)
        runs.append((linattn.scan_fwd(*[d[k] for k in PARAMS], S=Sd), Sd))
    within(runs[0][0], want["y"], rel(p, N, dtype) * size["y"], "y")
    within(runs[0][1], want["S"], (rel(p, N, "f32") + 2.0 ** -24) * size["S"], "S")
    for y, Sd in runs[1:]:
        assert torch.equal(y, runs[0][0]) and torch.equal(Sd, runs[0][1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [1.0, 200.0])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_live_nan_stays_in_the_state(cuda, linattn, dtype, decay, value):
    """What the recurrence makes of a row that is not a number: every later row of its column and the final
    state, even where the decay over the rest of the chunk is zero (0 times NaN); earlier chunks, other heads
    and other sequences are untouched, and so are the gradients' rows after the chunk."""
    B, N, H, G, D, M, at = 2, 420, 3, 1, 32, 16, 140
    p, dy, S = inputs(B, N, H, G, D, M, dtype, 8, decay)
    p["dt_bias"] = torch.zeros_like(p["dt_bias"])
    p["rows"][1, at, M + 5] = value  # x of head 1, column 5
    d = place(p, H, G, D, M, cuda)
    Sd = S.to(cuda)
    y = linattn.scan_fwd(*[d[k] for k in PARAMS], S=Sd)
    assert not torch.isfinite(y[1, at:, 1, 5]).any() and not torch.isfinite(Sd[1, 1, :, 5]).any()
    free = torch.ones_like(y, dtype=torch.bool)
    free[1, 128:, 1, 5] = False  # (its own chunk's earlier rows may hold it too)
    assert torch.isfinite(y[free]).all()
    free = torch.ones_like(Sd, dtype=torch.bool)
    free[1, 1, :, 5] = False
    assert torch.isfinite(Sd[free]).all()
    ddt, dA = (linattn.scan_bwd(*[d[k] for k in PARAMS], dy.to(cuda))[i] for i in (1, 2))
    assert not torch.isfinite(dA[1]) and torch.isfinite(dA[[0, 2]]).all()
    assert not torch.isfinite(ddt[1, at, 1]) and torch.isfinite(ddt[0]).all() and torch.isfinite(ddt[1, :, [0, 2]]).all()
