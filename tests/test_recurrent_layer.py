"""The operators together, as a decoder layer uses them: rows are convolved, scanned and then read an
encoder's states; a prompt is run at once and single tokens continue it; a training step and a decode
step are captured into CUDA graphs."""
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
