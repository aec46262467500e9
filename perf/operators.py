"""What is measured of the framework's recurrent layer: the short causal
convolution, the selective state space scan behind it, and the kernelized cross
attention to an encoder's states -- each over prompts, in training (forward and
gradients) and for single tokens.

``run`` computes a pass in its plain form (elementary torch operations in fp32,
fp64 for the long sums of log-decays) or, where ``own`` is true, by the
framework's calls.  Layouts: the scan's tensors are token-major, x [B, N, H, M],
dt [B, N, H], B and C [B, N, G, D], as views of the convolution's output rows
[x | B | C]; attention tensors are head-major, [B, H, N, D]; states are fp32,
[B, H, D, M].
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a training step's convolution over [x | B | C] rows of 32 heads of 64 and two groups of 64
        dict(name="conv train bf16", op="conv", how="train", B=4, N=2048, C=2304, K=4, dtype="bf16", ragged=False),
        # a ragged batch of prompts continuing from saved histories, fp32, a width of three
        dict(name="conv prompt f32 ragged", op="conv", how="prompt", B=3, N=1021, C=640, K=3, dtype="f32", ragged=True),
        # one token for each of 256 streams
        dict(name="conv step bf16", op="conv", how="step", B=256, N=1, C=2304, K=4, dtype="bf16", ragged=False),
        # two 4096-token prompts, every head sharing one B and C
        dict(name="scan prompt bf16", op="scan", how="prompt", B=2, N=4096, H=32, G=1, D=64, M=64, dtype="bf16", ragged=False),
        # one long prompt with few heads
        dict(name="scan prompt bf16 long", op="scan", how="prompt", B=1, N=65536, H=8, G=1, D=32, M=64, dtype="bf16", ragged=False),
        # a training step's scan
        dict(name="scan train bf16", op="scan", how="train", B=4, N=2048, H=32, G=2, D=64, M=64, dtype="bf16", ragged=False),
        # a small fp32 training step on padded 784-token images, B and C per head
        dict(name="scan train f32 ragged", op="scan", how="train", B=2, N=784, H=8, G=8, D=32, M=32, dtype="f32", ragged=True),
        # one token for each of 256 streams of 32 heads
        dict(name="scan step bf16", op="scan", how="step", B=256, N=1, H=32, G=1, D=64, M=64, dtype="bf16", ragged=False),
        # one stream of one small model: latency
        dict(name="scan step f32 one stream", op="scan", how="step", B=1, N=1, H=8, G=1, D=16, M=32, dtype="f32", ragged=False),
        # a decoder's training step over 2048-frame utterances of unequal lengths, grouped key heads
        dict(name="cross train bf16 ragged", op="cross", how="train", B=16, H=8, Hk=4, Nq=512, N=2048, D=64, M=64, dtype="bf16", ragged=True),
        # the same in fp32 at a small size, one key head for each query head
        dict(name="cross train f32 ragged", op="cross", how="train", B=4, H=6, Hk=6, Nq=201, N=800, D=32, M=64, dtype="f32", ragged=True),
        # one token for each of 2048 streams, read from the encoder's summed states
        dict(name="cross step bf16", op="cross", how="step", B=2048, H=8, Hk=8, Nq=1, N=0, D=64, M=64, dtype="bf16", ragged=False),
    ]


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 250


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op, dtype = rng.choice(("conv", "scan", "cross")), rng.choice(("bf16", "bf16", "f32"))
        how = rng.choice(("train", "prompt", "step"))
        if op == "conv":
            c = dict(op=op, how=how, B=_spread(rng, 1, 512 if how == "step" else 16), N=1 if how == "step" else _spread(rng, 1, 16384),
                     C=rng.choice((8 * _spread(rng, 8, 640), _spread(rng, 3, 5120))), K=rng.choice((2, 3, 4)), dtype=dtype, ragged=how != "step" and rng.random() < 0.5)
        elif op == "scan":
            h = _spread(rng, 1, 64)
            c = dict(op=op, how=how, B=_spread(rng, 1, 512 if how == "step" else 16), N=1 if how == "step" else _spread(rng, 1, 65536), H=h,
                     G=rng.choice([g for g in range(1, h + 1) if h % g == 0]), D=rng.choice((16, 32, 64)), M=rng.choice((16, 32, 64)),
                     dtype=dtype, ragged=how != "step" and rng.random() < 0.5)
        else:
            hk = _spread(rng, 1, 16)
            c = dict(op=op, how=how, B=_spread(rng, 1, 2048 if how == "step" else 32), H=hk * rng.choice((1, 1, 2, 3)), Hk=hk,
                     Nq=1 if how == "step" else _spread(rng, 1, 4096), N=0 if how == "step" else _spread(rng, 1, 16384),
                     D=rng.choice((16, 32, 64)), M=rng.choice((16, 32, 64)), dtype=dtype, ragged=how != "step" and rng.random() < 0.5)
        if _cost(c) <= most:
            return c


def _lengths(case, g):
    if not case["ragged"]:
        return None
    n = torch.randint(0, case["N"] + 1, (case["B"],), generator=g, device="cuda", dtype=torch.int32)
    n[0] = case["N"]  # a batch is padded to its longest sequence
    return n


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = DT[case["dtype"]]

    def normal(*shape, std=1.0, dtype=t):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case)
    B, N = case["B"], case["N"]
    s["lengths"] = _lengths(case, g)
    if case["op"] == "conv":
        C, K = case["C"], case["K"]
        wide = normal(B, N, C + 64)  # the projection's rows: [what is convolved | what is not]
        s["x"] = wide[..., :C] if case["how"] != "step" else wide[:, 0, :C]
        s["w"], s["bias"] = normal(C, K, std=K ** -0.5), normal(C, std=0.1)
        s["dy"] = normal(B, N, C) if case["how"] == "train" else None
        s["state"] = normal(B, K - 1, C) if case["how"] != "train" else None
    elif case["op"] == "scan":
        H, G, D, M = case["H"], case["G"], case["D"], case["M"]
        rows = normal(B, N, H * M + 2 * G * D)  # the convolution's output [x | B | C]
        x, b, c = rows.split([H * M, G * D, G * D], dim=-1)
        s["x"], s["Bm"], s["Cm"] = x.unflatten(-1, (H, M)), b.unflatten(-1, (G, D)), c.unflatten(-1, (G, D))
        s["dt"] = normal(B, N, H, std=0.5)
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))
        s["dt_bias"] = (step + torch.log(-torch.expm1(-step))).to(t)  # softplus(dt_bias) = step
        s["A"], s["skip"] = (-uniform(1.0, 16.0, H)).to(t), uniform(0.5, 1.5, H).to(t)
        s["dy"] = normal(B, N, H, M) if case["how"] == "train" else None
        s["S"] = normal(B, H, D, M, dtype=torch.float32) if case["how"] != "train" else None
        if case["how"] == "step":
            for n in ("x", "dt", "Bm", "Cm"):
                s[n] = s[n][:, 0]
    else:
        H, Hk, Nq, D, M = case["H"], case["Hk"], case["Nq"], case["D"], case["M"]
        s["q"] = normal(B, H, Nq, D) if case["how"] != "step" else normal(B, H, D)
        if case["how"] != "step":
            s["k"], s["v"] = normal(B, Hk, N, D), normal(B, Hk, N, M)
        else:  # an encoder of 1500 states, summed
            s["S"] = normal(B, Hk, D, M, std=1500 ** 0.5, dtype=torch.float32)
            s["Z"] = uniform(750.0, 2250.0, B, Hk, D)
        s["dout"] = normal(B, H, Nq, M) if case["how"] == "train" else None
    return s


# ------------------------------------------------------------- the plain forms

def _rows_mask(s, n):
    """[B, n] of which rows count, or None where all do."""
    return None if s["lengths"] is None else torch.arange(n, device="cuda")[None, :] < s["lengths"][:, None]


def _leaves(tensors, wanted):
    return [None if x is None else x.detach().float().requires_grad_(wanted) for x in tensors]


def _grads(y, dy, leaves, like):
    return [d.to(x.dtype) for d, x in zip(torch.autograd.grad(y, leaves, dy.float()), like)]


def _plain_conv(x, w, bias, history, mask):
    K, n = w.shape[1], x.shape[1]
    if mask is not None:
        x = torch.where(mask[..., None], x, 0.0)
    ext = torch.cat([history, x], 1)
    pre = bias + (ext.unfold(1, K, 1)[:, :n] * w).sum(-1)
    y = pre * torch.sigmoid(pre)
    return ext, y if mask is None else torch.where(mask[..., None], y, 0.0)


def _run_conv(s):
    x, w, bias, state = s["x"], s["w"], s["bias"], s["state"]
    K, t = w.shape[1], x.dtype
    if s["how"] == "step":
        ext = torch.cat([state.float(), x.float()[:, None]], 1)
        pre = bias.float() + (ext * w.float().t()[None]).sum(1)
        state.copy_(ext[:, 1:])
        return {"y": (pre * torch.sigmoid(pre)).to(t), "state": state}
    mask = _rows_mask(s, x.shape[1])
    if s["how"] == "prompt":
        ext, y = _plain_conv(x.float(), w.float(), bias.float(), state.float(), mask)
        n = torch.full((x.shape[0],), x.shape[1], device="cuda") if mask is None else s["lengths"].long()
        at = n[:, None] + torch.arange(K - 1, device="cuda")[None, :]
        state.copy_(ext.gather(1, at[..., None].expand(-1, -1, x.shape[2])))
        return {"y": y.to(t), "state": state}
    lx, lw, lb = _leaves((x, w, bias), True)
    with torch.enable_grad():
        _, y = _plain_conv(lx, lw, lb, torch.zeros_like(lx[:, :1]).expand(-1, K - 1, -1), mask)
    dx, dw, db = _grads(y, s["dy"], (lx, lw, lb), (x, w, bias))
    return {"y": y.detach().to(t), "dx": dx, "dw": dw, "db": db}


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _plain_scan(x, dt, A, Bm, Cm, skip, bias, S0, mask, T=64):
    """(y, state after the last row): chunks of T rows, each chunk's pairs as a masked
    matrix, the chunks' states joined through a matrix of the decays between chunks."""
    b, n, H, M = x.shape
    G, D = Bm.shape[2:]
    c = -(-n // T)
    delta = _softplus(dt + bias)
    if mask is not None:
        delta = torch.where(mask[..., None], delta, 0.0)
        x, Bm = torch.where(mask[..., None, None], x, 0.0), torch.where(mask[..., None, None], Bm, 0.0)

    def cut(v):  # [b, n, h, ...] -> [b, h, chunk, T, ...]
        v = torch.nn.functional.pad(v, [0, 0] * (v.dim() - 2) + [0, c * T - n])
        return v.unflatten(1, (c, T)).movedim(3, 1)

    u = cut(x * delta[..., None])
    kb, kc = (cut(v.repeat_interleave(H // G, 2)) for v in (Bm, Cm))
    cum = torch.cumsum(cut((delta.double() * A.double())[..., None])[..., 0], -1)  # [b, H, c, T]
    low = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
    pairs = torch.exp(torch.where(low, cum[..., :, None] - cum[..., None, :], -math.inf)).float()
    y = (pairs * (kc @ kb.transpose(-1, -2))) @ u
    own_state = (kb * torch.exp(cum[..., -1:] - cum).float()[..., None]).transpose(-1, -2) @ u  # [b, H, c, D, M]
    total = torch.nn.functional.pad(torch.cumsum(cum[..., -1], -1), (1, 0))  # [b, H, c + 1]
    before = torch.ones(c + 1, c + 1, dtype=torch.bool, device="cuda").tril()
    hops = torch.exp(torch.where(before, total[..., :, None] - total[..., None, :], -math.inf)).float()
    start = torch.zeros_like(own_state[:, :, :1]) if S0 is None else S0[:, :, None]
    states = (hops @ torch.cat([start, own_state], 2).flatten(3)).unflatten(3, (D, M))
    y = y + (kc * torch.exp(cum).float()[..., None]) @ states[:, :, :-1]
    y = y.movedim(1, 3).flatten(1, 2)[:, :n] + x * skip[:, None]
    return y if mask is None else torch.where(mask[..., None, None], y, 0.0), states[:, :, -1]


def _run_scan(s):
    x, names = s["x"], ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias")
    t = x.dtype
    if s["how"] == "step":
        xf, dt, A, Bm, Cm, skip, bias = (s[n].float() for n in names)
        H, G = xf.shape[1], Bm.shape[1]
        Bm, Cm = Bm.repeat_interleave(H // G, 1), Cm.repeat_interleave(H // G, 1)
        delta = _softplus(dt + bias)
        s["S"].mul_(torch.exp(delta * A)[..., None, None]).add_(Bm[..., None] * (delta[..., None] * xf)[..., None, :])
        y = (Cm[..., None] * s["S"]).sum(-2) + skip[:, None] * xf
        return {"y": y.to(t), "S": s["S"]}
    mask = _rows_mask(s, x.shape[1])
    if s["how"] == "prompt":
        y, S = _plain_scan(*(s[n].float() for n in names), s["S"], mask)
        s["S"].copy_(S)
        return {"y": y.to(t), "S": s["S"]}
    leaves = _leaves([s[n] for n in names], True)
    with torch.enable_grad():
        y, _ = _plain_scan(*leaves, None, mask)
    grads = _grads(y, s["dy"], leaves, [s[n] for n in names])
    return {"y": y.detach().to(t), **{"d" + n: d for n, d in zip(names, grads)}}


def _phi(x):
    return torch.where(x > 0, x + 1.0, torch.exp(torch.clamp(x, max=0.0)))


def _plain_cross(q, k, v, mask):
    fk = _phi(k)
    if mask is not None:
        fk, v = torch.where(mask[:, None, :, None], fk, 0.0), torch.where(mask[:, None, :, None], v, 0.0)
    S, Z = fk.transpose(-1, -2) @ v, fk.sum(2)
    out, den = _plain_read(q, S, Z)
    return out, den, S, Z


def _plain_read(q, S, Z):
    r = q.shape[1] // S.shape[1]
    fq, S, Z = _phi(q), S.repeat_interleave(r, 1), Z.repeat_interleave(r, 1)
    den = (fq * Z[:, :, None]).sum(-1)
    some = den > 0  # a sequence of no states gives zeros
    return torch.where(some[..., None], fq @ S / torch.where(some, den, 1.0)[..., None], 0.0), den


def _run_cross(s):
    q = s["q"]
    if s["how"] == "step":
        return {"y": _plain_read(q.float()[:, :, None], s["S"], s["Z"])[0][:, :, 0].to(q.dtype)}
    k, v = s["k"], s["v"]
    mask = _rows_mask(s, k.shape[2])
    if s["how"] == "prompt":
        out, den, S, Z = _plain_cross(q.float(), k.float(), v.float(), mask)
        return {"out": out.to(q.dtype), "den": den, "S": S, "Z": Z}
    lq, lk, lv = _leaves((q, k, v), True)
    with torch.enable_grad():
        out, den, S, Z = _plain_cross(lq, lk, lv, mask)
    dq, dk, dv = _grads(out, s["dout"], (lq, lk, lv), (q, k, v))
    return {"out": out.detach().to(q.dtype), "den": den.detach(), "S": S.detach(), "Z": Z.detach(), "dq": dq, "dk": dk, "dv": dv}


# --------------------------------------------------------- the framework's calls

def _own(s):
    import kernelized_causal_attention_gb300 as la
    n = s["lengths"]
    if s["op"] == "conv":
        a = (s["x"], s["w"], s["bias"])
        if s["how"] == "step":
            return {"y": la.short_conv_step(*a, s["state"]), "state": s["state"]}
        if s["how"] == "prompt":
            return {"y": la.short_conv_fwd(*a, state=s["state"], lengths=n), "state": s["state"]}
        y = la.short_conv_fwd(*a, lengths=n)
        dx, dw, db = la.short_conv_bwd(*a, s["dy"], lengths=n)
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    if s["op"] == "scan":
        names = ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias")
        a = [s[k] for k in names]
        if s["how"] == "step":
            return {"y": la.scan_step(*a, s["S"]), "S": s["S"]}
        if s["how"] == "prompt":
            return {"y": la.scan_fwd(*a, S=s["S"], lengths=n), "S": s["S"]}
        y = la.scan_fwd(*a, lengths=n)
        return {"y": y, **{"d" + k: d for k, d in zip(names, la.scan_bwd(*a, s["dy"], lengths=n))}}
    if s["how"] == "step":
        return {"y": la.cross_step(s["q"], s["S"], s["Z"])}
    out, den, S, Z = la.cross_fwd(s["q"], s["k"], s["v"], n)
    got = {"out": out, "den": den, "S": S, "Z": Z}
    if s["how"] == "train":
        got["dq"], got["dk"], got["dv"] = la.cross_bwd(s["q"], s["k"], s["v"], n, out, den, S, Z, s["dout"])
    return got


def run(state):
    if own:
        return _own(state)
    return {"conv": _run_conv, "scan": _run_scan, "cross": _run_cross}[state["op"]](state)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, N, how = case["B"], case["N"], case["how"]
    if case["op"] == "conv":
        C, K = case["C"], case["K"]
        row, tap = B * N * C, C * (K + 1)
        if how == "train":  # x, dy read; y, dx written; the taps and their gradients
            return {"bytes": e * (4 * row + 2 * tap), "flops": row * (6 * K + 12)}
        return {"bytes": e * (2 * row + tap + 2 * B * (K - 1) * C), "flops": row * (2 * K + 4)}
    D, M, H = case["D"], case["M"], case["H"]
    if case["op"] == "scan":
        G = case["G"]
        rows = B * N * (H * M + 2 * G * D + H)  # x, B, C, dt
        if how == "train":  # read by the forward pass and by the backward, where the gradients are written
            return {"bytes": e * (2 * rows + rows + 2 * B * N * H * M), "flops": B * N * H * (14 * D * M + 10 * M)}
        return {"bytes": e * (rows + B * N * H * M) + 8 * B * H * D * M, "flops": B * N * H * (5 * D * M + 4 * M)}
    Hk, Nq = case["Hk"], case["Nq"]
    if how == "step":
        return {"bytes": e * B * H * (D + M) + 4 * B * Hk * (D * M + D), "flops": B * H * 2 * D * M}
    once = e * (B * H * Nq * (D + M) + B * Hk * N * (D + M)) + 4 * (B * H * Nq + B * Hk * D * (M + 1))
    flops = 2 * D * M * B * (H * Nq + Hk * N)
    if how == "prompt":
        return {"bytes": once, "flops": flops}
    more = e * (B * H * Nq * (2 * D + 2 * M) + B * Hk * N * 2 * (D + M)) + 4 * (B * H * Nq + B * Hk * D * (M + 1))
    return {"bytes": once + more, "flops": 3 * flops}


# ------------------------------------------------- the definitions, in 64 bits

def _exact_conv(s):
    x, w, bias = s["x"].double(), s["w"].double(), s["bias"].double()
    K = w.shape[1]
    if s["how"] == "step":
        x = x[:, None]
    b, n, C = x.shape
    lengths = [n] * b if s["lengths"] is None else s["lengths"].tolist()
    old = torch.zeros(b, K - 1, C, device="cuda", dtype=torch.double) if s["state"] is None else s["state"].double()
    y, dx, new = torch.zeros_like(x), torch.zeros_like(x), old.clone()
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for i, m in enumerate(lengths):
        ext = torch.cat([old[i], x[i, :m]])
        new[i] = ext[m:]
        if m == 0:
            continue
        pre = bias + sum(ext[j:j + m] * w[:, j] for j in range(K))
        sig = 1 / (1 + torch.exp(-pre))
        y[i, :m] = pre * sig
        if s["dy"] is not None:
            g = s["dy"][i, :m].double() * sig * (1 + pre * (1 - sig))
            db += g.sum(0)
            for j in range(K):
                dw[:, j] += (g * ext[j:j + m]).sum(0)
                back = K - 1 - j  # tap j reaches from row t to row t - back
                if m > back:
                    dx[i, :m - back] += g[back:] * w[:, j]
    if s["how"] == "train":
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    return {"y": y[:, 0] if s["how"] == "step" else y, "state": new}


def _exact_scan(s):
    names = ("x", "dt", "A", "Bm", "Cm", "skip", "dt_bias")
    x, dt, A, Bm, Cm, skip, bias = (s[n].double() for n in names)
    if s["how"] == "step":
        x, dt, Bm, Cm = (v[:, None] for v in (x, dt, Bm, Cm))
    b, n, H, M = x.shape
    G, D = Bm.shape[2:]
    z = dt + bias
    delta = torch.logaddexp(z, torch.zeros_like(z))
    live = torch.ones(b, n, device="cuda", dtype=torch.bool) if s["lengths"] is None else torch.arange(n, device="cuda") < s["lengths"][:, None]
    delta = delta * live[..., None]
    a = torch.exp(delta * A)
    Bh, Ch = Bm.repeat_interleave(H // G, 2), Cm.repeat_interleave(H // G, 2)
    S = torch.zeros(b, H, D, M, device="cuda", dtype=torch.double) if s["S"] is None else s["S"].double()
    train = s["how"] == "train"
    u = delta[..., None] * x
    y, kept = torch.empty_like(x), []
    for t in range(n):
        if train:
            kept.append(S)
        S = a[:, t, :, None, None] * S + Bh[:, t, :, :, None] * u[:, t, :, None, :]
        y[:, t] = torch.einsum("bhd,bhdm->bhm", Ch[:, t], S)
    y = (y + skip[:, None] * x) * live[..., None, None]
    if not train:
        return {"y": y[:, 0] if s["how"] == "step" else y, "S": S}
    dy = s["dy"].double() * live[..., None, None]
    du, dBh, dCh, dl = torch.empty_like(x), torch.empty_like(Bh), torch.empty_like(Ch), torch.empty_like(delta)
    R = torch.zeros_like(S)
    for t in range(n - 1, -1, -1):
        R = R + Ch[:, t, :, :, None] * dy[:, t, :, None, :]
        dCh[:, t] = torch.einsum("bhdm,bhm->bhd", S, dy[:, t])
        S = kept.pop()
        du[:, t] = torch.einsum("bhd,bhdm->bhm", Bh[:, t], R)
        dBh[:, t] = torch.einsum("bhdm,bhm->bhd", R, u[:, t])
        R = a[:, t, :, None, None] * R
        dl[:, t] = (R * S).sum((2, 3))
    ddelta = ((du * x).sum(-1) + A * dl) * live[..., None]
    dz = ddelta / (1 + torch.exp(-z))
    got = (delta[..., None] * du + skip[:, None] * dy, dz, (delta * dl).sum((0, 1)), dBh.unflatten(2, (G, H // G)).sum(3),
           dCh.unflatten(2, (G, H // G)).sum(3), (dy * x).sum((0, 1, 3)), dz.sum((0, 1)))
    return {"y": y, **{"d" + k: d for k, d in zip(names, got)}}


def _exact_cross(s):
    if s["how"] == "step":
        q, S, Z = s["q"].double(), s["S"].double(), s["Z"].double()
        r = q.shape[1] // S.shape[1]
        fq = torch.where(q > 0, q + 1, torch.exp(q.clamp(max=0)))
        y = torch.stack([torch.einsum("bd,bdm->bm", fq[:, h], S[:, h // r]) / (fq[:, h] * Z[:, h // r]).sum(-1, keepdim=True)
                         for h in range(q.shape[1])], 1)
        return {"y": y}
    r, found = s["H"] // s["Hk"], []
    lengths = [s["N"]] * s["B"] if s["lengths"] is None else s["lengths"].tolist()
    for i, m in enumerate(lengths):  # every pair of a query and a state, one sequence and key head at a time
        for h in range(s["Hk"]):
            q, k, v = s["q"][i, h * r:(h + 1) * r].double(), s["k"][i, h].double(), s["v"][i, h].double()
            fq, fk = (torch.where(a > 0, a + 1, torch.exp(a.clamp(max=0))) for a in (q, k[:m]))
            w = fq @ fk.t()  # [r, Nq, m]
            den = w.sum(-1)
            out = w @ v[:m] / den[..., None] if m else torch.zeros(*q.shape[:2], v.shape[1], device="cuda", dtype=torch.double)
            got = {"out": out, "den": den, "S": (fk.t() @ v[:m])[None], "Z": fk.sum(0)[None]}
            if s["how"] == "train":
                dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
                if m:
                    d = s["dout"][i, h * r:(h + 1) * r].double() / den[..., None]
                    dw = d @ v[:m].t() - (d * out).sum(-1, keepdim=True)
                    dq = dw @ fk * torch.where(q > 0, 1.0, fq)
                    dk[:m] = torch.einsum("rqm,rqd->md", dw, fq) * torch.where(k[:m] > 0, 1.0, fk)
                    dv[:m] = torch.einsum("rqm,rqn->mn", w, d)
                got |= {"dq": dq, "dk": dk[None], "dv": dv[None]}
            found.append(got)
    return {n: torch.stack([torch.cat([g[n] for g in found[i * s["Hk"]:(i + 1) * s["Hk"]]]) for i in range(s["B"])]) for n in found[0]}


def exact(case, seed):
    if case["op"] == "scan" and case["how"] == "train" and 8 * case["N"] * case["B"] * case["H"] * case["D"] * case["M"] > 60e9:
        return None  # the recurrence keeps every row's state
    if case["op"] == "cross" and case["B"] * case["H"] * case["Nq"] * case["N"] * (case["D"] + case["M"]) > 1e12:
        return None  # every pair, in 64 bits
    return {"conv": _exact_conv, "scan": _exact_scan, "cross": _exact_cross}[case["op"]](prepare(case, seed))
