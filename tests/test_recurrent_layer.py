"""The operators together, as a decoder layer uses them: rows are convolved, scanned and then read an
encoder's states; a prompt is run at once and single tokens continue it; a training step and a decode
step are captured into CUDA graphs."""
import threading

import pytest
import torch

import kernelized_causal_attention_gb300 as la
import plain64
from plain64 import BF16, within

pytestmark = pytest.mark.gpu

B, N, H, G, D, M, K, NE = 3, 150, 4, 2, 32, 64, 4, 90
C = H * M + 2 * G * D


def layer(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).bfloat16()  # noqa: E731
    w = {"w": r(C, K), "b": r(C), "A": -1 - r(H).abs(), "skip": r(H), "dt_bias": r(H) - 2}
    return w, r(B, N, C + H), r(B, 2, NE, D), r(B, 2, NE, M), torch.tensor([90, 0, 31], dtype=torch.int32)


def cut(rows):
    """[x | B | C] of the convolution's output, in place."""
    x, b, c = rows.split([H * M, G * D, G * D], dim=-1)
    return x.unflatten(-1, (H, M)), b.unflatten(-1, (G, D)), c.unflatten(-1, (G, D))


def queries(y):
    """The scan's heads as the cross attention's queries (head-major, the first D columns)."""
    return y[..., :D].transpose(1, 2).contiguous()


def test_prompt_then_tokens_is_the_whole(cuda):
    w, rows, k, v, n = layer()
    wd = {a: t.to(cuda) for a, t in w.items()}
    rows, k, v, n = rows.to(cuda), k.to(cuda), v.to(cuda), n.to(cuda)

    def prompt(rows, hist, S):
        u = la.short_conv_fwd(rows[..., :C], wd["w"], wd["b"], state=hist)
        x, b, c = cut(u)
        return u, la.scan_fwd(x, rows[..., C:], wd["A"], b, c, wd["skip"], wd["dt_bias"], S=S)

    new = lambda: (torch.zeros(B, K - 1, C, dtype=torch.bfloat16, device=cuda), torch.zeros(B, H, D, M, device=cuda))  # noqa: E731
    hist, S = new()
    u, y = prompt(rows, hist, S)
    out, _, SE, ZE = la.cross_fwd(queries(y), k, v, n)
    hist2, S2 = new()
    split = 140
    _, y0 = prompt(rows[:, :split].contiguous(), hist2, S2)
    ys, outs = [y0], [la.cross_fwd(queries(y0), k, v, n)[0]]
    for t in range(split, N):
        ut = la.short_conv_step(rows[:, t, :C], wd["w"], wd["b"], hist2)
        x, b, c = cut(ut)
        yt = la.scan_step(x, rows[:, t, C:], wd["A"], b, c, wd["skip"], wd["dt_bias"], S2)
        ys.append(yt[:, None])
        outs.append(la.cross_step(yt[..., :D].contiguous(), SE, ZE)[:, :, None])
    assert torch.equal(hist, hist2)
    # against the 64-bit scan on the same convolved rows, and the 64-bit attention on the same queries
    x, b, c = cut(u.cpu())
    args = (x, rows[..., C:].cpu(), w["A"], b, c, w["skip"], w["dt_bias"])
    want, size = plain64.scan(*args), plain64.scan(*args, size=True)
    for got in (y, torch.cat(ys, 1)):
        within(got, want["y"], 2.1 * BF16 * size["y"], "y")
    for got in (S, S2):
        within(got, want["S"], 2.0 ** -15 * size["S"], "S")
    q = queries(torch.cat(ys, 1))
    want, size = plain64.cross(q, k, v, n.tolist()), plain64.cross(q, k, v, n.tolist(), size=True)
    within(torch.cat(outs, 2), want["out"], 3.2 * BF16 * size["out"], "out")
    assert torch.isfinite(out).all() and float(out[1].abs().max()) == 0.0
    la.check_device_status()


def test_training_step_in_a_graph(cuda):
    """Forward and gradients of the whole layer, captured once and replayed on new inputs, equal the
    eager calls bit for bit; eager gradients are taken again after the capture."""
    w, rows, k, v, n = layer(1)
    wd = {a: t.to(cuda) for a, t in w.items()}
    rows, k, v, n = rows.to(cuda), k.to(cuda), v.to(cuda), n.to(cuda)
    dout = torch.randn(B, H, N, M, device=cuda).bfloat16()

    def step():
        u = la.short_conv_fwd(rows[..., :C], wd["w"], wd["b"])
        x, b, c = cut(u)
        dt = rows[..., C:]
        y = la.scan_fwd(x, dt, wd["A"], b, c, wd["skip"], wd["dt_bias"])
        q = queries(y)
        out, den, S, Z = la.cross_fwd(q, k, v, n)
        dq, dk, dv = la.cross_bwd(q, k, v, n, out, den, S, Z, dout)
        dy = torch.zeros_like(y)
        dy[..., :D] = dq.transpose(1, 2)
        dx, ddt, dA, dB, dC, ds, db = la.scan_bwd(x, dt, wd["A"], b, c, wd["skip"], wd["dt_bias"], dy)
        du = torch.cat([dx.flatten(2), dB.flatten(2), dC.flatten(2)], -1)
        drows, dw, dbias = la.short_conv_bwd(rows[..., :C], wd["w"], wd["b"], du)
        return [out, dk, dv, ddt, dA, ds, db, drows, dw, dbias]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = step()
    for seed in (2, 3):
        rows.copy_(layer(seed)[1])
        graph.replay()
        replayed = [t.clone() for t in held]
        for a, b in zip(replayed, step()):
            assert torch.equal(a, b) and torch.isfinite(a).all()
    la.check_device_status()


def test_autograd_of_the_layer(cuda):
    """The autograd functions, chained, give what the calls give."""
    w, rows, k, v, n = layer(4)
    rows = rows.to(cuda).requires_grad_(True)
    p = {a: t.to(cuda).requires_grad_(True) for a, t in w.items()}
    k, v, n = k.to(cuda).requires_grad_(True), v.to(cuda).requires_grad_(True), n.to(cuda)
    u = la.short_conv(rows[..., :C], p["w"], p["b"])
    x, b, c = cut(u)
    y = la.selective_scan(x, rows[..., C:], p["A"], b, c, p["skip"], p["dt_bias"])
    out = la.cross_linear_attention(y[..., :D].transpose(1, 2), k, v, n)
    dout = torch.randn(out.shape, device=cuda).bfloat16()
    grads = torch.autograd.grad(out, [rows, k, v, *p.values()], dout)
    q = queries(y.detach())
    f = la.cross_fwd(q, k.detach(), v.detach(), n)
    dq, dk, dv = la.cross_bwd(q, k.detach(), v.detach(), n, *f, dout)
    assert torch.equal(grads[1], dk) and torch.equal(grads[2], dv)
    dy = torch.zeros_like(y)
    dy[..., :D] = dq.transpose(1, 2)
    back = la.scan_bwd(x.detach(), rows.detach()[..., C:], p["A"].detach(), b.detach(), c.detach(), p["skip"].detach(), p["dt_bias"].detach(), dy)
    for g, want in zip(grads[5:], (back[2], back[5], back[6])):
        assert torch.equal(g, want)
    assert torch.equal(grads[0][..., C:], back[1])
    assert all(torch.isfinite(g).all() for g in grads)


def test_two_streams_at_once(cuda):
    """Two layers' scans on two streams at the same time, each with its own workspace."""
    w, rows, *_ = layer(5)
    wd = {a: t.to(cuda) for a, t in w.items()}
    ins = [layer(s)[1].to(cuda) for s in (6, 7)]
    x = [cut(r[..., :C].contiguous()) for r in ins]
    run = lambda i: la.scan_fwd(x[i][0], ins[i][..., C:], wd["A"], x[i][1], x[i][2], wd["skip"], wd["dt_bias"])  # noqa: E731
    want = [run(0), run(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(i))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g, want[i])


def test_back_to_back_with_the_causal_kernels(cuda):
    """The causal attention's kernels and these, launched one behind the other without a wait: every
    kernel may start while the one before it ends, and both take tensor memory."""
    w, rows, k, v, n = layer(8)
    wd = {a: t.to(cuda) for a, t in w.items()}
    rows, k, v = rows.to(cuda), k.to(cuda), v.to(cuda)
    x, b, c = cut(rows[..., :C].contiguous())
    dt, dy = rows[..., C:], torch.randn(B, N, H, M, device=cuda).bfloat16()
    q, kk, vv = (torch.randn(2, 4, 700, 64, device=cuda).bfloat16() for _ in range(3))

    def once():
        out, den = la.causal_fwd(q, kk, vv)
        y = la.scan_fwd(x, dt, wd["A"], b, c, wd["skip"], wd["dt_bias"])
        f = la.cross_fwd(queries(y), k, v)
        grads = la.causal_bwd(q, kk, vv, out, den, vv)
        back = la.scan_bwd(x, dt, wd["A"], b, c, wd["skip"], wd["dt_bias"], dy)
        out2, _ = la.causal_fwd(q, kk, vv)
        return [out, y, *f, *grads, *back, *la.cross_bwd(queries(y), k, v, None, *f, f[0]), out2]

    want = once()
    torch.cuda.synchronize()
    runs = [once() for _ in range(12)]
    torch.cuda.synchronize()
    for r in runs:
        for a, t in zip(r, want):
            assert torch.equal(a, t)
    la.check_device_status()


def test_first_call_of_a_host_thread(cuda):
    """A host thread that has made no CUDA call yet (as an autograd engine's before its first gradient)
    has no context of its own; every raw entry point works as its first call."""
    w, rows, k, v, n = layer(9)
    wd = {a: t.to(cuda) for a, t in w.items()}
    rows, k, v = rows.to(cuda)[..., :C].contiguous(), k.to(cuda), v.to(cuda)
    x, b, c = cut(rows)
    dt = torch.randn(B, N, H, device=cuda).bfloat16()
    y = la.scan_fwd(x, dt, wd["A"], b, c)
    q = queries(y)
    f = la.cross_fwd(q, k, v)
    scan, cross = (B, H, G, N, D, M), (B, H, 2, N, NE, D, M)
    ld = (C, H, C, C)
    new = lambda *ts: [torch.full_like(t, float("nan")) for t in ts]  # noqa: E731
    room = lambda n: torch.empty(n, dtype=torch.uint8, device=cuda)  # noqa: E731
    s_ws = [room(la.la_scan_workspace_bytes(i, *scan, la.LA_BF16)) for i in (0, 1)]
    c_ws = [room(la.la_cross_workspace_bytes(i, *cross, la.LA_BF16)) for i in (0, 1)]
    conv_ws = room(la.la_short_conv_workspace_bytes(B, N, C, K, la.LA_BF16))
    none = None
    back = la.scan_bwd(x, dt, wd["A"], b, c, none, none, y)
    cback = la.cross_bwd(q, k, v, none, *f, f[0])
    conv, conv_back = la.short_conv_fwd(rows, wd["w"], wd["b"]), la.short_conv_bwd(rows, wd["w"], wd["b"], rows)
    outs = {"scan_fwd": new(y), "scan_bwd": new(*back[:5]), "cross_fwd": new(*f), "cross_bwd": new(*cback), "conv_fwd": new(conv), "conv_bwd": new(*conv_back)}
    stream = torch.cuda.current_stream().cuda_stream
    a = [torch.randn(2, 4, 300, 64, device=cuda).bfloat16() for _ in range(3)]
    causal, causal_ws = la.causal_fwd(*a), la.workspace(la.LA_OP_CAUSAL_FWD, 2, 4, 300, 64, 64, la.LA_BF16, cuda)
    outs["causal_fwd"] = new(*causal)
    o = outs
    calls = {
        "scan_fwd": lambda: la.la_scan_fwd(x, dt, wd["A"], b, c, none, none, none, none, *o["scan_fwd"], s_ws[0], *scan, *ld, la.LA_BF16, stream),
        "scan_bwd": lambda: la.la_scan_bwd(x, dt, wd["A"], b, c, none, none, none, y, *o["scan_bwd"], none, none, s_ws[1], *scan, *ld, la.LA_BF16, stream),
        "cross_fwd": lambda: la.la_cross_fwd(q, k, v, none, *o["cross_fwd"], c_ws[0], *cross, la.LA_BF16, stream),
        "cross_bwd": lambda: la.la_cross_bwd(q, k, v, none, *f, f[0], *o["cross_bwd"], c_ws[1], *cross, la.LA_BF16, stream),
        "conv_fwd": lambda: la.la_short_conv_fwd(rows, wd["w"], wd["b"], none, none, *o["conv_fwd"], B, N, C, K, C, 1, la.LA_BF16, stream),
        "conv_bwd": lambda: la.la_short_conv_bwd(rows, wd["w"], wd["b"], none, rows, *o["conv_bwd"], conv_ws, B, N, C, K, C, 1, la.LA_BF16, stream),
    }
    calls["causal_fwd"] = lambda: la.la_causal_fwd(*a, *o["causal_fwd"], causal_ws, 2, 4, 300, 64, 64, la.LA_BF16, stream)
    failed = {}

    def first(name):
        try:
            calls[name]()
        except Exception as e:  # noqa: BLE001
            failed[name] = repr(e)

    for name in calls:
        t = threading.Thread(target=first, args=(name,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not failed
    want = {"scan_fwd": [y], "scan_bwd": back[:5], "cross_fwd": f, "cross_bwd": cback, "conv_fwd": [conv], "conv_bwd": conv_back, "causal_fwd": causal}
    for name, got in outs.items():
        for u, t in zip(got, want[name]):
            assert torch.equal(u, t), name


def test_decode_step_in_a_graph(cuda):
    """One token of the whole layer, captured once: replays on new rows go through the same histories and states as the
    eager calls, bit for bit."""
    w, rows, k, v, n = layer(10)
    wd = {a: t.to(cuda) for a, t in w.items()}
    rows, k, v, n = rows.to(cuda), k.to(cuda), v.to(cuda), n.to(cuda)
    _, _, SE, ZE = la.cross_fwd(torch.zeros(B, H, 1, D, dtype=torch.bfloat16, device=cuda), k, v, n)
    new = lambda: (torch.zeros(B, K - 1, C, dtype=torch.bfloat16, device=cuda), torch.zeros(B, H, D, M, device=cuda))  # noqa: E731

    def step(row, hist, S):
        u = la.short_conv_step(row[:, :C], wd["w"], wd["b"], hist)
        x, b, c = cut(u)
        y = la.scan_step(x, row[:, C:], wd["A"], b, c, wd["skip"], wd["dt_bias"], S)
        return la.cross_step(y[..., :D].contiguous(), SE, ZE)

    row, (hist, S) = rows[:, 0].clone(), new()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(row, hist, S)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step(row, hist, S)
    hist.zero_(), S.zero_()
    hist2, S2 = new()
    for t in range(12):
        row.copy_(rows[:, t])
        graph.replay()
        assert torch.equal(out, step(rows[:, t], hist2, S2)) and torch.isfinite(out).all()
    assert torch.equal(hist, hist2) and torch.equal(S, S2)
    la.check_device_status()
