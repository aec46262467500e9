"""The operators around the recurrent layer together, as a model uses them: rows are normalised behind a residual sum,
convolved, run through the gated recurrence, read as rotated keys and queries of the scan, normalised by heads, and
a token reads an encoder's packed states; a prompt at once and single tokens after it, a training step, graphs,
streams, views and threads."""
import inspect
import threading

import pytest
import torch

import around64
import kernelized_causal_attention_gb300 as la
from around64 import rounded
from plain64 import within

B, N, H, G, D, M, K = 3, 150, 4, 2, 32, 16, 4
C = H * M  # the gated recurrence's channels are the scan's heads


def layer(dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = dict(w=1 + 0.1 * r(3 * C), b=0.1 * r(3 * C), taps=0.5 * r(3 * C, K), lam=-6 + r(C), A=-torch.rand(H, generator=g), hw=1 + 0.1 * r(C))
    return {n: t.to(dtype) for n, t in p.items()}, r(B, N, 3 * C).to(dtype), r(B, N, 3 * C).to(dtype), r(B, N, 2 * G * D + H).to(dtype)


def to(dev, *ts):
    return [t.to(dev) if isinstance(t, torch.Tensor) else {n: u.to(dev) for n, u in t.items()} for t in ts]


def split3(u):
    return u[..., :C], u[..., C:2 * C], u[..., 2 * C:3 * C]


def keys(kq):
    """k, q and dt as slices of one row."""
    k, q, dt = kq[..., :G * D], kq[..., G * D:2 * G * D], kq[..., 2 * G * D:]
    return k.unflatten(-1, (G, D)), q.unflatten(-1, (G, D)), dt


def prompt(p, rows, res, kq, turns, hist, h, S, positions, n=None):
    y0, s, _, _ = la.norm_fwd(rows, p["w"], p["b"], residual=res, lengths=n)
    u = la.short_conv_fwd(y0, p["taps"], state=hist, lengths=n)
    v = la.gated_fwd(*split3(u), p["lam"], h=h, lengths=n)
    k, q, dt = keys(kq)
    q, k = la.rotary_fwd(q, k, turns, positions=positions, lengths=n)
    o = la.scan_fwd(v.unflatten(-1, (H, M)), dt, p["A"], k, q, S=S, lengths=n)
    return dict(y0=y0, s=s, u=u, v=v, q=q, k=k, o=o, out=la.norm_fwd(o.flatten(2), p["hw"], groups=H, lengths=n)[0])


def token(p, rows, res, kq, turns, hist, h, S, positions):
    y0, s, _, _ = la.norm_fwd(rows, p["w"], p["b"], residual=res)
    u = la.short_conv_step(y0, p["taps"], None, hist)
    v = la.gated_step(*split3(u), p["lam"], h)
    k, q, dt = keys(kq)
    q, k = la.rotary_fwd(q, k, turns, positions=positions)
    o = la.scan_step(v.unflatten(-1, (H, M)), dt, p["A"], k, q, None, None, S)
    return dict(y0=y0, s=s, u=u, v=v, q=q, k=k, o=o, out=la.norm_fwd(o.flatten(1), p["hw"], groups=H)[0])


def states(dtype, dev):
    return torch.zeros(B, K - 1, 3 * C, dtype=dtype, device=dev), torch.zeros(B, C, device=dev), torch.zeros(B, H, D, M, device=dev)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_then_tokens_is_the_whole(cuda, linattn, dtype):
    """A prompt of 140 rows and ten tokens: every stage within its bounds of the 64-bit form over the whole sequence, given
    the rows that the stage before it made."""
    p, rows, res, kq = layer(dtype)
    pd, rd, sd, kd = to(cuda, p, rows, res, kq)
    turns, _ = la.rotary_turns(D, device=cuda)
    exact = [t % (1 << 64) for t in turns.tolist()]
    start = torch.tensor([0, 5, 1 << 20], dtype=torch.int32)
    hist, h, S = states(dtype, cuda)
    cut = 140
    first = prompt(pd, rd[:, :cut].contiguous(), sd[:, :cut].contiguous(), kd[:, :cut].contiguous(), turns, hist, h, S, start.to(cuda))
    whole = {n: [t] for n, t in first.items()}
    for t in range(cut, N):
        for n, v in token(pd, rd[:, t], sd[:, t], kd[:, t], turns, hist, h, S, (start + t).to(cuda)).items():
            whole[n].append(v[:, None])
    got = {n: torch.cat(v, 1).cpu() for n, v in whole.items()}
    name = "f32" if dtype == torch.float32 else "bf16"
    want = around64.norm(rows, p["w"], p["b"], res)
    within(got["y0"], want["y"][0], rounded(*want["y"], name), "norm")
    assert torch.equal(got["s"].double(), want["s"][0])
    hist2, h2, S2 = states(dtype, cuda)
    u = la.short_conv_fwd(got["y0"].to(cuda), pd["taps"], state=hist2)
    assert torch.equal(u.cpu(), got["u"]) and torch.equal(hist, hist2)
    want = around64.gated(*split3(got["u"]), p["lam"])
    within(got["v"], want["y"][0], rounded(*want["y"], name), "gated recurrence")
    within(h, want["h"][0], want["h"][1], "its state")
    at = start[:, None].long() + torch.arange(N)
    for n, x in zip("kq", keys(kq)):
        want, e = around64.rotary(x, exact, at)
        within(got[n], want, rounded(want, e, name), n)
    want = around64.norm(got["o"].flatten(2), p["hw"], groups=H)["y"]
    within(got["out"], want[0], rounded(*want, name), "norm by heads")
    o = la.scan_fwd(got["v"].to(cuda).unflatten(-1, (H, M)), kd[..., -H:], pd["A"], got["k"].to(cuda), got["q"].to(cuda), S=S2)
    size = float(o.double().abs().max())
    assert float((o.cpu().double() - got["o"].double()).abs().max()) <= (1e-5 if name == "f32" else 2e-2) * size
    assert float((S - S2).abs().max()) <= 1e-5 * float(S2.abs().max())
    la.check_device_status()


@pytest.mark.gpu
def test_a_ragged_batch_is_its_sequences(cuda, linattn):
    """Padded rows hold NaN; every sequence and its states are, bit for bit, what a batch without padding gives."""
    p, rows, res, kq = to(cuda, *layer(torch.bfloat16, 1))
    n = torch.tensor([N, 0, 77], dtype=torch.int32, device=cuda)
    turns, _ = la.rotary_turns(D, device=cuda)
    clean = states(torch.bfloat16, cuda)
    want = prompt(p, rows, res, kq, turns, *clean, None, n)
    for t in (rows, res, kq):
        t[1], t[2, 77:] = float("nan"), float("nan")
    got_states = states(torch.bfloat16, cuda)
    got = prompt(p, rows, res, kq, turns, *got_states, None, n)
    for name in want:
        assert torch.equal(got[name], want[name]), name
        assert float(got[name][1].abs().max()) == 0.0 and float(got[name][2, 77:].abs().max()) == 0.0
    for a, b in zip(got_states, clean):
        assert torch.equal(a, b)


def training(p, rows, res, kq, turns, dout):
    y0, s, mean, rstd = la.norm_fwd(rows, p["w"], p["b"], residual=res)
    u = la.short_conv_fwd(y0, p["taps"])
    v, kept = la.gated_fwd(*split3(u), p["lam"], keep=True)
    k, q, dt = keys(kq)
    q, k = la.rotary_fwd(q, k, turns)
    x = v.unflatten(-1, (H, M))
    o = la.scan_fwd(x, dt, p["A"], k, q)
    out, _, m2, r2 = la.norm_fwd(o.flatten(2), p["hw"], groups=H)
    do, dhw, _ = la.norm_bwd(o.flatten(2), p["hw"], m2, r2, dout, groups=H, bias=False)
    dx, ddt, dA, dk, dq, _, _ = la.scan_bwd(x, dt, p["A"], k, q, None, None, do.unflatten(-1, (H, M)))
    dq, dk = la.rotary_bwd(dq, dk, turns)
    dv, dr, di, dlam = la.gated_bwd(*split3(u), p["lam"], kept, dx.flatten(2))
    du = torch.cat([dv, dr, di], -1)
    dy0, dtaps, _ = la.short_conv_bwd(y0, p["taps"], None, du)
    drows, dw, db = la.norm_bwd(s, p["w"], mean, rstd, dy0, dy0)
    return [out, s, drows, dw, db, dtaps, dlam, dA, dhw, torch.cat([dk.flatten(2), dq.flatten(2), ddt], -1)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_autograd_of_the_layer(cuda, linattn, dtype):
    """The autograd functions, chained, give what the calls give."""
    p, rows, res, kq = to(cuda, *layer(dtype, 2))
    turns, _ = la.rotary_turns(D, device=cuda)
    dout = torch.randn(B, N, C, device=cuda).to(dtype)
    want = training(p, rows, res, kq, turns, dout)
    leaves = [t.clone().requires_grad_(True) for t in (rows, res, kq, *p.values())]
    rows, res, kq = leaves[:3]
    q = dict(zip(p, leaves[3:]))
    y0, s = la.layer_norm(rows, q["w"], q["b"], res)
    u = la.short_conv(y0, q["taps"])
    v = la.gated_recurrence(*split3(u), q["lam"])
    k, qq, dt = keys(kq)
    qq, k = la.rotary(qq, k, turns)
    o = la.selective_scan(v.unflatten(-1, (H, M)), dt, q["A"], k, qq)
    out = la.layer_norm(o.flatten(2), q["hw"], groups=H)
    assert torch.equal(out, want[0]) and torch.equal(s, want[1])
    grads = torch.autograd.grad((out, s), leaves, (dout, torch.zeros_like(s)), allow_unused=True)
    # `training` sends the gradient of y0 into s as well: here nothing reaches s by another way
    du = torch.cat(la.gated_bwd(*split3(u.detach()), p["lam"], la.gated_fwd(*split3(u.detach()), p["lam"], keep=True)[1], _dv(p, v, kq, turns, dout))[:3], -1)
    dy0 = la.short_conv_bwd(y0.detach(), p["taps"], None, du)[0]
    base = la.norm_bwd(s.detach(), p["w"], *la.norm_fwd(rows.detach(), p["w"], p["b"], residual=res.detach())[2:], dy0)
    for a, b in zip(grads, (base[0], base[0], want[9], base[1], base[2], want[5], want[6], want[7], want[8])):
        assert torch.equal(a, b) and torch.isfinite(a).all()


def _dv(p, v, kq, turns, dout):
    """The gradient that reaches the gated recurrence's output."""
    k, q, dt = keys(kq.detach())
    q, k = la.rotary_fwd(q, k, turns)
    x = v.detach().unflatten(-1, (H, M))
    o = la.scan_fwd(x, dt, p["A"], k, q)
    _, _, m, r = la.norm_fwd(o.flatten(2), p["hw"], groups=H)
    do = la.norm_bwd(o.flatten(2), p["hw"], m, r, dout, groups=H, bias=False)[0]
    return la.scan_bwd(x, dt, p["A"], k, q, None, None, do.unflatten(-1, (H, M)))[0].flatten(2)


def capture(f, s=None):
    s = s or torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = f()
    return graph, held


@pytest.mark.gpu
def test_training_step_in_a_graph(cuda, linattn):
    """Captured once and replayed on new inputs: the eager calls' results bit for bit, before and after them."""
    p, rows, res, kq = to(cuda, *layer(torch.bfloat16, 3))
    turns, _ = la.rotary_turns(D, device=cuda)
    dout = torch.randn(B, N, C, device=cuda).bfloat16()
    step = lambda: training(p, rows, res, kq, turns, dout)  # noqa: E731
    graph, held = capture(step)
    for seed in (4, 5):
        _, a, b, c = to(cuda, *layer(torch.bfloat16, seed))
        rows.copy_(a), res.copy_(b), kq.copy_(c)
        graph.replay()
        replayed = [t.clone() for t in held]
        for x, y in zip(replayed, step()):
            assert torch.equal(x, y) and torch.isfinite(x).all()
    la.check_device_status()


@pytest.mark.gpu
def test_token_in_a_graph_with_packed_states(cuda, linattn):
    """One token of the layer and its read of the packed encoder, captured: replays go through the eager calls' states."""
    p, rows, res, kq = to(cuda, *layer(torch.bfloat16, 6))
    turns, _ = la.rotary_turns(D, device=cuda)
    k, v = torch.randn(B, G, 60, 16, device=cuda).bfloat16(), torch.randn(B, G, 60, 32, device=cuda).bfloat16()
    _, _, SE, ZE = la.cross_fwd(torch.zeros(B, H, 1, 16, dtype=torch.bfloat16, device=cuda), k, v)
    codes, scale = la.state_pack(SE)
    row, other, keys_, at = rows[:, 0].clone(), res[:, 0].clone(), kq[:, 0].clone(), torch.zeros(B, dtype=torch.int32, device=cuda)
    st = states(torch.bfloat16, cuda)

    def step(row, other, keys_, at, st):
        out = token(p, row, other, keys_, turns, *st, at)["out"]
        return la.cross_step_packed(out.unflatten(-1, (H, M)).contiguous(), codes, scale, ZE)

    graph, held = capture(lambda: step(row, other, keys_, at, st))
    for t in st:
        t.zero_()
    st2 = states(torch.bfloat16, cuda)
    for t in range(12):
        row.copy_(rows[:, t]), other.copy_(res[:, t]), keys_.copy_(kq[:, t]), at.fill_(t)
        graph.replay()
        want = step(rows[:, t], res[:, t], kq[:, t], torch.full_like(at, t), st2)
        assert torch.equal(held, want) and torch.isfinite(held).all()
    for a, b in zip(st, st2):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_two_streams_and_two_graphs_at_once(cuda, linattn):
    """Two training steps on two streams, eager and as two graphs, at the same time."""
    ins = [to(cuda, *layer(torch.bfloat16, s)) for s in (7, 8)]
    turns, _ = la.rotary_turns(D, device=cuda)
    dout = torch.randn(B, N, C, device=cuda).bfloat16()
    run = [lambda a=a: training(*a, turns, dout) for a in ins]
    want = [f() for f in run]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = [capture(f, s) for f, s in zip(run, streams)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run[i]())
                graphs[i][0].replay()
    torch.cuda.synchronize()
    for i in range(2):
        for g in (*got[i], graphs[i][1]):
            for a, b in zip(g, want[i]):
                assert torch.equal(a, b)
    la.check_device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", ["gated", "norm", "rotary"])
def test_gradient_at_an_odd_address(cuda, linattn, name, dtype):
    """A result behind others in one vector: its gradient is a dense view that starts one element in."""
    g = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(s, generator=g).to(dtype).to(cuda).requires_grad_(True)  # noqa: E731
    turns, _ = la.rotary_turns(4, device=cuda)
    f, leaves = {"gated": (la.gated_recurrence, [r(1, 3, 5), r(1, 3, 5), r(1, 3, 5), r(5)]), "norm": (la.layer_norm, [r(1, 3, 5), r(5), r(5)]),
                 "rotary": (lambda x: la.rotary(x, None, turns)[0], [r(1, 3, 1, 5)])}[name]
    y = f(*leaves)
    d = torch.randn(y.numel() + 1, device=cuda).to(dtype)
    want = torch.autograd.grad(f(*leaves), leaves, d[1:].clone().view(y.shape))
    got = torch.autograd.grad(torch.cat([torch.zeros(1, dtype=dtype, device=cuda), y.flatten()]), leaves, d)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # and an expanded one, as a sum's backward gives
    got = torch.autograd.grad(f(*leaves).float().sum(), leaves)
    want = torch.autograd.grad(f(*leaves), leaves, torch.ones_like(y))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_first_call_of_a_host_thread(cuda, linattn):
    p, rows, res, kq = to(cuda, *layer(torch.bfloat16, 10))
    turns, _ = la.rotary_turns(D, device=cuda)
    dout = torch.randn(B, N, C, device=cuda).bfloat16()
    want, got = training(p, rows, res, kq, turns, dout), []
    torch.cuda.synchronize()
    t = threading.Thread(target=lambda: got.extend(training(p, rows, res, kq, turns, dout)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def cpu_arguments():
    z = torch.zeros
    x, lam, kept = z(2, 5, 8), z(8), z(2 * 8)
    rows = dict(x=x, r=x, i=x, lam=lam)
    q, t = z(2, 5, 4, 16), z(8, dtype=torch.int64)
    codes = z(1, 1, 16, 32, dtype=torch.int8)
    return {
        "gated_fwd": rows, "gated_bwd": dict(rows, kept=kept, dy=x), "gated_step": {**{n: x[:, 0] for n in "xri"}, "lam": lam, "h": z(2, 8)},
        "norm_fwd": dict(x=x, w=lam), "norm_bwd": dict(s=x, w=lam, mean=z(2, 5, 1), rstd=z(2, 5, 1), dy=x),
        "rotary_fwd": dict(q=q, k=q, turns=t), "rotary_bwd": dict(dq=q, dk=q, turns=t),
        "state_pack": dict(S=z(1, 1, 16, 32)), "state_unpack": dict(codes=codes, scale=z(1, 1, 16)),
        "cross_step_packed": dict(q=z(1, 2, 16), codes=codes, scale=z(1, 1, 16), Z=z(1, 1, 16)),
    }


@pytest.mark.parametrize("name", sorted(cpu_arguments()))
def test_by_keyword(linattn, name):
    """Every argument by its documented name: the call gets as far as asking for a CUDA device."""
    f, kw = getattr(linattn, name), cpu_arguments()[name]
    assert set(kw) <= set(inspect.signature(f).parameters)
    with pytest.raises(ValueError, match="CUDA device"):
        f(**kw)
    first = next(iter(kw))
    with pytest.raises(TypeError, match=first):
        f(**{n: t for n, t in kw.items() if n != first})
