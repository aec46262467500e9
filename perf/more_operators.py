"""What is measured of the operators around the recurrent layer: the gated
recurrence (a decay and a state for each channel), the layer norm with its
residual sum and its form by heads, rotary positions, and 8-bit packed states --
over prompts, in training (forward and gradients) and for single tokens.

``run`` computes a pass in its plain form (elementary torch operations in fp32,
fp64 for the angles of positions) or, where ``own`` is true, by the framework's
calls.  Layouts: rows are token-major, [B, N, C] and [B, N, H, D] (rotary also
head-major, [B, H, N, D]), as views of wider rows where a projection writes them
side by side; states are fp32, [B, C] and [B, H, D, M].
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"i8": 127.0, "e4m3": 448.0}
SCALE = 8.0  # the gated recurrence's factor of softplus(lam)
EPS = 1e-5


def listed():
    return [
        # a training step's recurrence over rows as wide as 32 heads of 64
        dict(name="gated train bf16", op="gated", how="train", B=4, N=2048, C=2048, dtype="bf16", ragged=False),
        # one long prompt of a narrow layer, continuing from a state
        dict(name="gated prompt bf16 long", op="gated", how="prompt", B=1, N=65536, C=512, dtype="bf16", ragged=False),
        # a small fp32 training step on padded images, an odd width
        dict(name="gated train f32 ragged", op="gated", how="train", B=3, N=784, C=645, dtype="f32", ragged=True),
        # one token for each of 256 streams
        dict(name="gated step bf16", op="gated", how="step", B=256, N=1, C=2048, dtype="bf16", ragged=False),
        # a training step's norm behind a residual sum, one weight a model channel
        dict(name="norm train bf16 residual", op="norm", how="train", B=4, N=2048, C=2048, G=1, residual=True, dtype="bf16", ragged=False),
        # the scan's output normalised head by head
        dict(name="norm train bf16 heads", op="norm", how="train", B=4, N=2048, C=2048, G=32, residual=False, dtype="bf16", ragged=False),
        # small padded fp32 rows of an odd width: latency
        dict(name="norm train f32 ragged", op="norm", how="train", B=2, N=131, C=777, G=1, residual=True, dtype="f32", ragged=True),
        # a training step's queries and keys, sixteen heads on four, out of one projection's rows
        dict(name="rotary train bf16", op="rotary", how="train", B=4, N=2048, H=16, Hk=4, D=64, R=64, pairs="half", layout="rows", scaled=1.0, dtype="bf16", ragged=False),
        # a long prompt, head-major, half of each head, frequencies stretched for eight times the length
        dict(name="rotary prompt f32 long", op="rotary", how="prompt", B=1, N=65536, H=8, Hk=8, D=64, R=32, pairs="adjacent", layout="heads", scaled=8.0, dtype="f32", ragged=False),
        # one token for each of 256 streams at positions up to a million
        dict(name="rotary step bf16", op="rotary", how="step", B=256, N=1, H=8, Hk=2, D=64, R=64, pairs="adjacent", layout="rows", scaled=1.0, dtype="bf16", ragged=False),
        # one token for each of 2048 streams, read from 8-bit states
        dict(name="packed step bf16 i8", op="packed", how="step", B=2048, H=8, Hk=8, D=64, M=64, code="i8", dtype="bf16"),
        # a batch of decode states put away in 8 bits and taken up again
        dict(name="packed park e4m3", op="packed", how="park", B=100, H=6, Hk=6, D=32, M=64, code="e4m3", dtype="f32"),
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
        op, dtype = rng.choice(("gated", "norm", "rotary", "packed")), rng.choice(("bf16", "bf16", "f32"))
        how = rng.choice(("train", "prompt", "step"))
        B, N = (_spread(rng, 1, 512), 1) if how == "step" else (_spread(rng, 1, 16), _spread(rng, 1, 65536))
        c = dict(op=op, how=how, B=B, N=N, dtype=dtype, ragged=how != "step" and rng.random() < 0.5)
        if op == "gated":
            c["C"] = rng.choice((8 * _spread(rng, 8, 640), _spread(rng, 3, 5120)))
        elif op == "norm":
            c["G"] = rng.choice((1, 1, _spread(rng, 2, 64)))
            width = (8 * _spread(rng, 2, 1024), _spread(rng, 1, 8192)) if c["G"] == 1 else (16, 32, 64, 64, _spread(rng, 1, 300))
            c["C"] = c["G"] * rng.choice(width)
            c["residual"] = rng.random() < 0.5
        elif op == "rotary":
            c["Hk"] = _spread(rng, 1, 16)
            c["H"] = c["Hk"] * rng.choice((1, 1, 2, 4))
            c["D"] = rng.choice((16, 32, 64, 64, 128, _spread(rng, 2, 256)))
            c["R"] = 2 * rng.choice((c["D"] // 2, max(1, c["D"] // 4), rng.randint(1, c["D"] // 2)))
            c["pairs"], c["layout"], c["scaled"] = rng.choice(("half", "adjacent")), rng.choice(("rows", "heads")), rng.choice((1.0, 1.0, 4.0, 8.0))
        else:
            c = dict(op=op, how=rng.choice(("step", "step", "park")), B=_spread(rng, 1, 2048), Hk=_spread(rng, 1, 16), D=rng.choice((16, 32, 64)),
                     M=rng.choice((16, 32, 64)), code=rng.choice(("i8", "e4m3")), dtype=dtype)
            c["H"] = c["Hk"] * (1 if c["how"] == "park" else rng.choice((1, 1, 2, 3)))
        if _cost(c) <= most:
            return c


def _lengths(case, g):
    if not case["ragged"]:
        return None
    n = torch.randint(0, case["N"] + 1, (case["B"],), generator=g, device="cuda", dtype=torch.int32)
    n[0] = case["N"]  # a batch is padded to its longest sequence
    return n


def _frequencies(R, factor):
    """Radians a position for each of R / 2 pairs, and the rotation's gain.  A factor above one stretches
    the slow pairs (those of less than one turn in 2048 positions) by it, leaves the fast ones (more than
    32 turns) alone and goes over between the two."""
    freq = [10000.0 ** (-2.0 * j / R) for j in range(R // 2)]
    if factor == 1.0:
        return freq, 1.0
    ramp = [min(1.0, max(0.0, (2048 * f / (2 * math.pi) - 1) / 31)) for f in freq]
    return [f * (w + (1 - w) / factor) for f, w in zip(freq, ramp)], 0.1 * math.log(factor) + 1


def _pack(S, code):
    """(codes, scale): every row of M values in 8 bits, by its largest magnitude."""
    scale = S.abs().amax(-1) / torch.full((), TOP[code], device="cuda")
    q = S / torch.where(scale > 0, scale, 1.0)[..., None]
    return (q.round().to(torch.int8) if code == "i8" else q.to(torch.float8_e4m3fn)), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = DT[case["dtype"]]

    def normal(*shape, std=1.0, dtype=t):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case)
    B, how = case["B"], case["how"]
    if case["op"] == "packed":
        H, Hk, D, M = case["H"], case["Hk"], case["D"], case["M"]
        S = normal(B, Hk, D, M, std=1500 ** 0.5, dtype=torch.float32)  # 1500 rows, summed
        if how == "park":
            s["S"] = S
        else:
            s["q"], s["Z"] = normal(B, H, D), uniform(750.0, 2250.0, B, Hk, D)
            s["codes"], s["scale"] = _pack(S, case["code"])
        return s
    N = case["N"]
    s["lengths"] = _lengths(case, g)
    if case["op"] == "gated":
        C = case["C"]
        s["x"] = normal(B, N, C)  # the convolution's output
        s["r"], s["i"] = normal(B, N, 2 * C).split(C, -1)  # both gates of one projection
        rate = -torch.log(uniform(0.9, 0.999, C)) / SCALE  # a of an open gate
        s["lam"] = torch.log(torch.expm1(rate)).to(t)
        s["dy"] = normal(B, N, C) if how == "train" else None
        s["h"] = normal(B, C, dtype=torch.float32) if how != "train" else None
        if how == "step":
            for n in ("x", "r", "i"):
                s[n] = s[n][:, 0]
    elif case["op"] == "norm":
        C = case["C"]
        s["x"] = (torch.randn((B, N, C), generator=g, device="cuda") + uniform(-0.5, 0.5, C)).to(t)
        s["w"], s["b"] = uniform(0.5, 1.5, C).to(t), normal(C, std=0.1)
        s["residual"] = normal(B, N, C, std=2.0) if case["residual"] else None
        s["dy"] = normal(B, N, C) if how == "train" else None
        s["ds"] = normal(B, N, C) if how == "train" and case["residual"] else None
    else:
        H, Hk, D, R = case["H"], case["Hk"], case["D"], case["R"]
        if case["layout"] == "rows":  # one projection's rows [q | k | v]
            q, k, _ = normal(B, N, (H + 2 * Hk) * D).split([H * D, Hk * D, Hk * D], -1)
            s["q"], s["k"] = q.unflatten(-1, (H, D)), k.unflatten(-1, (Hk, D))
            s["dq"], s["dk"] = (normal(B, N, H, D), normal(B, N, Hk, D)) if how == "train" else (None, None)
        else:
            s["q"], s["k"] = normal(B, H, N, D), normal(B, Hk, N, D)
            s["dq"], s["dk"] = (normal(B, H, N, D), normal(B, Hk, N, D)) if how == "train" else (None, None)
        freq, s["gain"] = _frequencies(R, case["scaled"])
        s["freq"] = torch.tensor(freq, device="cuda", dtype=torch.float64)
        s["turns"] = torch.tensor([round(f / (2 * math.pi) * 2.0 ** 64) for f in freq], device="cuda")
        # training starts at zero, a prompt goes on somewhere, a stream's token is anywhere
        far = 1 << 20 if how == "step" else 8192
        s["start"] = None if how == "train" else torch.randint(0, far, (B,), generator=g, device="cuda", dtype=torch.int32)
    return s


# ------------------------------------------------------------- the plain forms

def _rows_mask(s, n):
    """[B, n] of which rows count, or None where all do."""
    return None if s["lengths"] is None else torch.arange(n, device="cuda")[None, :] < s["lengths"][:, None]


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _gates(s):
    """(decay exponent u, a, beta, sigmoid(r), sigmoid(i)) in fp32."""
    sr, gi = torch.sigmoid(s["r"].float()), torch.sigmoid(s["i"].float())
    u = SCALE * _softplus(s["lam"].float()) * sr
    return u, torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u)), sr, gi


def _recurrence(a, b):
    """h_n = a_n h_{n-1} + b_n along the rows, by doubling."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return a, b


def _run_gated(s):
    x, t = s["x"].float(), s["x"].dtype
    u, a, beta, sr, gi = _gates(s)
    if s["how"] == "step":
        s["h"].mul_(a).add_(beta * gi * x)
        return {"y": s["h"].to(t), "h": s["h"]}
    mask = _rows_mask(s, x.shape[1])
    b = beta * gi * x
    if mask is not None:
        mask = mask[..., None]
        a, b = torch.where(mask, a, 1.0), torch.where(mask, b, 0.0)
    if s["how"] == "prompt":
        total, h = _recurrence(a, b)
        h = h + total * s["h"][:, None]
        s["h"].copy_(h[:, -1])
        return {"y": (h if mask is None else torch.where(mask, h, 0.0)).to(t), "h": s["h"]}
    h = _recurrence(a, b)[1]
    dy = s["dy"].float() if mask is None else torch.where(mask, s["dy"].float(), 0.0)
    ahead = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)  # the decay of the row after
    G = _recurrence(ahead.flip(1), dy.flip(1))[1].flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    Q = a * G * (a * gi * x * torch.where(u > 0, u / beta, 0.0) - u * before)
    if mask is not None:
        G, Q, h = torch.where(mask, G, 0.0), torch.where(mask, Q, 0.0), torch.where(mask, h, 0.0)
    lam = s["lam"].float()
    dlam = torch.sigmoid(lam) / _softplus(lam) * Q.sum((0, 1))
    return {"y": h.to(t), "dx": (G * beta * gi).to(t), "dr": (Q * (1 - sr)).to(t), "di": (G * beta * x * gi * (1 - gi)).to(t), "dlam": dlam.to(t)}


def _run_norm(s):
    x, t, G = s["x"], s["x"].dtype, s["G"]
    mask = _rows_mask(s, x.shape[1])
    total = x if s["residual"] is None else (x.float() + s["residual"].float()).to(t)
    v = total.float().unflatten(-1, (G, -1))
    w, b = s["w"].float().unflatten(-1, (G, -1)), s["b"].float().unflatten(-1, (G, -1))
    v = v - v.mean(-1, keepdim=True)
    rstd = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    xh = v * rstd

    def live(z):
        z = z.flatten(2)
        return (z if mask is None else torch.where(mask[..., None], z, torch.zeros_like(z))).to(t)

    out = {"y": live(xh * w + b)}
    if s["residual"] is not None:
        out["s"] = live(total.unflatten(-1, (G, -1)))
    if s["how"] != "train":
        return out
    dy = s["dy"].float() if mask is None else torch.where(mask[..., None], s["dy"].float(), 0.0)
    dy = dy.unflatten(-1, (G, -1))
    dxh = dy * w
    d = (dxh - dxh.mean(-1, keepdim=True) - xh * (dxh * xh).mean(-1, keepdim=True)) * rstd
    if s["ds"] is not None:
        d = d + s["ds"].float().unflatten(-1, (G, -1))
    out["dx"] = live(d)
    out["dw"], out["db"] = (dy * xh).sum((0, 1)).flatten().to(t), dy.sum((0, 1)).flatten().to(t)
    return out


def _turn(x, cos, sin, s, mask):
    """The rotation of x [B, N, H, D] (or head-major), with cos and sin [B, N, R / 2]."""
    R, heads = s["R"], s["layout"] == "heads"
    at = 1 if heads else 2
    cos, sin = cos.unsqueeze(at), sin.unsqueeze(at)
    f = x.float()
    a, b = (f[..., :R // 2], f[..., R // 2:R]) if s["pairs"] == "half" else (f[..., 0:R:2], f[..., 1:R:2])
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([p, q], -1) if s["pairs"] == "half" else torch.stack([p, q], -1).flatten(-2)
    y = torch.cat([turned, f[..., R:]], -1)
    if mask is not None:
        y = torch.where((mask.unsqueeze(at))[..., None], y, 0.0)
    return y.to(x.dtype)


def _run_rotary(s):
    names = ("q", "k")
    if s["how"] == "step":
        n, mask = 1, None
    else:
        n = s["N"]
        mask = _rows_mask(s, n)
    at = torch.arange(n, device="cuda")[None, :] + (0 if s["start"] is None else s["start"][:, None])
    angle = at.expand(s["B"], n)[..., None].double() * s["freq"]
    cos, sin = (torch.cos(angle) * s["gain"]).float(), (torch.sin(angle) * s["gain"]).float()
    got = {m: _turn(s[m], cos, sin, s, mask) for m in names}
    if s["how"] == "train":
        got |= {"d" + m: _turn(s["d" + m], cos, -sin, s, mask) for m in names}
    return got


def _phi(x):
    return torch.where(x > 0, x + 1.0, torch.exp(torch.clamp(x, max=0.0)))


def _run_packed(s):
    if s["how"] == "park":
        codes, scale = _pack(s["S"], s["code"])
        return {"S": codes.float() * scale[..., None], "scale": scale}
    q, r = s["q"], s["H"] // s["Hk"]
    fq = _phi(q.float()).unflatten(1, (s["Hk"], r))
    S = s["codes"].float() * s["scale"][..., None]
    y = (fq @ S) / (fq * s["Z"][:, :, None]).sum(-1, keepdim=True)
    return {"y": y.flatten(1, 2).to(q.dtype)}


# --------------------------------------------------------- the framework's calls

def _own(s):
    import kernelized_causal_attention_gb300 as la
    if s["op"] == "packed":
        if s["how"] == "park":
            codes, scale = la.state_pack(s["S"], CODE[s["code"]])
            return {"S": la.state_unpack(codes, scale), "scale": scale}
        return {"y": la.cross_step_packed(s["q"], s["codes"], s["scale"], s["Z"])}
    n = s["lengths"]
    if s["op"] == "gated":
        a = (s["x"], s["r"], s["i"], s["lam"])
        if s["how"] == "step":
            return {"y": la.gated_step(*a, s["h"], scale=SCALE), "h": s["h"]}
        if s["how"] == "prompt":
            return {"y": la.gated_fwd(*a, h=s["h"], scale=SCALE, lengths=n), "h": s["h"]}
        y, kept = la.gated_fwd(*a, scale=SCALE, lengths=n, keep=True)
        dx, dr, di, dlam = la.gated_bwd(*a, kept, s["dy"], scale=SCALE, lengths=n)
        return {"y": y, "dx": dx, "dr": dr, "di": di, "dlam": dlam}
    if s["op"] == "norm":
        y, total, mean, rstd = la.norm_fwd(s["x"], s["w"], s["b"], residual=s["residual"], groups=s["G"], eps=EPS, lengths=n)
        out = {"y": y} if s["residual"] is None else {"y": y, "s": total}
        if s["how"] == "train":
            out["dx"], out["dw"], out["db"] = la.norm_bwd(total, s["w"], mean, rstd, s["dy"], ds=s["ds"], groups=s["G"], lengths=n)
        return out
    how = dict(positions=s["start"], gain=s["gain"], interleaved=s["pairs"] == "adjacent", head_major=s["layout"] == "heads", lengths=n)
    q, k = la.rotary_fwd(s["q"], s["k"], s["turns"], **how)
    out = {"q": q, "k": k}
    if s["how"] == "train":
        out["dq"], out["dk"] = la.rotary_bwd(s["dq"], s["dk"], s["turns"], **how)
    return out


def run(state):
    if own:
        return _own(state)
    return {"gated": _run_gated, "norm": _run_norm, "rotary": _run_rotary, "packed": _run_packed}[state["op"]](state)


def work(case):
    e, B, how = 2 if case["dtype"] == "bf16" else 4, case["B"], case["how"]
    if case["op"] == "packed":
        state = B * case["Hk"] * case["D"]
        if how == "park":  # the state read, its codes and scales written, read, and the state written
            return {"bytes": state * (10 * case["M"] + 8), "flops": 4 * state * case["M"]}
        return {"bytes": state * (case["M"] + 8) + e * B * case["H"] * (case["D"] + case["M"]), "flops": B * case["H"] * 2 * case["D"] * case["M"]}
    rows = B * case["N"]
    if case["op"] == "gated":
        n = rows * case["C"]
        if how == "train":  # x, r, i read by the forward pass and by the backward, which reads dy and writes three gradients
            return {"bytes": e * (11 * n + 3 * case["C"]), "flops": 90 * n}
        return {"bytes": e * (4 * n + case["C"]) + 8 * B * case["C"], "flops": 35 * n}
    if case["op"] == "norm":
        n, more = rows * case["C"], 2 if case["residual"] else 0
        if how == "train":  # with a residual, its sum is written and its own gradient read
            return {"bytes": e * ((5 + more + (1 if more else 0)) * n + 5 * case["C"]), "flops": 25 * n}
        return {"bytes": e * ((2 + more) * n + 2 * case["C"]), "flops": 8 * n}
    n = rows * (case["H"] + case["Hk"])
    once = {"bytes": e * 2 * n * case["D"] + 4 * case["R"], "flops": 3 * n * case["R"]}
    return {k: v * (2 if how == "train" else 1) for k, v in once.items()}


# ------------------------------------------------- the definitions, in 64 bits

def _exact_gated(s):
    x, r, i, lam = (s[n].double() for n in ("x", "r", "i", "lam"))
    if s["how"] == "step":
        x, r, i = x[:, None], r[:, None], i[:, None]
    B, N, C = x.shape
    live = torch.ones(B, N, 1, device="cuda", dtype=torch.bool) if s["lengths"] is None else (torch.arange(N, device="cuda") < s["lengths"][:, None])[..., None]
    soft = torch.logaddexp(lam, torch.zeros_like(lam))
    sr, gi = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
    a = torch.exp(-SCALE * soft * sr)
    beta = torch.sqrt(-torch.expm1(-2 * SCALE * soft * sr))
    keep, put = torch.where(live, a, 1.0), torch.where(live, beta * gi * x, 0.0)
    h = torch.zeros(B, C, device="cuda", dtype=torch.double) if s["h"] is None else s["h"].double()
    y, before = torch.empty_like(x), torch.empty_like(x)
    for n in range(N):
        before[:, n] = h
        h = keep[:, n] * h + put[:, n]
        y[:, n] = h
    y = torch.where(live, y, 0.0)
    if s["how"] != "train":
        return {"y": y[:, 0] if s["how"] == "step" else y, "h": h}
    G, grad = torch.zeros(B, C, device="cuda", dtype=torch.double), torch.empty_like(x)
    dy = torch.where(live, s["dy"].double(), 0.0)
    for n in range(N - 1, -1, -1):
        G = G + dy[:, n]
        grad[:, n] = G
        G = keep[:, n] * G
    dbeta = grad * gi * x
    da = grad * before - dbeta * a / torch.where(beta > 0, beta, 1.0)
    dlog = torch.where(live, da * a, 0.0)  # with respect to log a = -scale softplus(lam) sigmoid(r)
    dsr = -SCALE * soft * dlog
    dlam = (-SCALE * sr * dlog).sum((0, 1)) / (1 + torch.exp(-lam))
    return {"y": y, "dx": torch.where(live, grad * beta * gi, 0.0), "dr": dsr * sr * (1 - sr),
            "di": torch.where(live, grad * beta * x, 0.0) * gi * (1 - gi), "dlam": dlam}


def _exact_norm(s):
    x, t, G = s["x"], s["x"].dtype, s["G"]
    B, N, C = x.shape
    M = C // G
    total = x.double() if s["residual"] is None else (x.double() + s["residual"].double()).to(t).double()  # the sum is kept in the rows' type
    w, b = s["w"].double(), s["b"].double()
    lengths = [N] * B if s["lengths"] is None else s["lengths"].tolist()
    y, dx, dw, db = torch.zeros_like(total), torch.zeros_like(total), torch.zeros_like(w), torch.zeros_like(w)
    kept = torch.zeros_like(total)
    for i, n in enumerate(lengths):
        kept[i, :n] = total[i, :n]
        for g in range(G):
            c = slice(g * M, (g + 1) * M)
            v = total[i, :n, c]
            var, m = torch.var_mean(v, -1, correction=0, keepdim=True)
            sd = torch.sqrt(var + EPS)
            z = (v - m) / sd
            y[i, :n, c] = z * w[c] + b[c]
            if s["how"] == "train":
                d = s["dy"][i, :n, c].double()
                dw[c] += (d * z).sum(0)
                db[c] += d.sum(0)
                d = d * w[c]
                dx[i, :n, c] = (d - (d.sum(-1, keepdim=True) + z * (d * z).sum(-1, keepdim=True)) / M) / sd
        if s["ds"] is not None:
            dx[i, :n] += s["ds"][i, :n].double()
    out = {"y": y} if s["residual"] is None else {"y": y, "s": kept}
    return out if s["how"] != "train" else out | {"dx": dx, "dw": dw, "db": db}


def _exact_rotary(s):
    R, N = s["R"], s["N"]
    first = torch.zeros(s["B"], device="cuda", dtype=torch.double) if s["start"] is None else s["start"].double()
    phase = torch.polar(torch.full((), s["gain"], device="cuda", dtype=torch.double).expand(s["B"], N, R // 2).contiguous(),
                        (first[:, None] + torch.arange(N, device="cuda"))[..., None] * s["freq"])
    live = torch.ones(s["B"], N, device="cuda", dtype=torch.bool) if s["lengths"] is None else torch.arange(N, device="cuda") < s["lengths"][:, None]

    def turned(x, phase):
        x = x.double() if s["layout"] == "rows" else x.double().transpose(1, 2)
        y = x.clone()
        pairs = torch.complex(*((x[..., :R // 2], x[..., R // 2:R]) if s["pairs"] == "half" else (x[..., 0:R:2], x[..., 1:R:2])))
        z = pairs * phase[:, :, None]
        if s["pairs"] == "half":
            y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
        else:
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
        y = y * live[:, :, None, None]
        return y if s["layout"] == "rows" else y.transpose(1, 2)

    out = {n: turned(s[n], phase) for n in ("q", "k")}
    return out | {n: turned(s[n], phase.conj()) for n in ("dq", "dk")} if s["how"] == "train" else out


def _exact_packed(s):
    if s["how"] == "park":  # the scale is an fp32 number, and so is the quotient that a code rounds
        S, f32 = s["S"].double(), torch.float32
        scale = (S.abs().amax(-1) / TOP[s["code"]]).to(f32).double()
        q = (S / scale[..., None]).to(f32)
        codes = torch.round(q).double() if s["code"] == "i8" else q.to(torch.float8_e4m3fn).double()
        return {"S": codes * scale[..., None], "scale": scale}
    q, Z, r = s["q"].double(), s["Z"].double(), s["H"] // s["Hk"]
    fq = torch.where(q > 0, q + 1, torch.exp(q.clamp(max=0)))
    S = s["codes"].double() * s["scale"].double()[..., None]
    return {"y": torch.stack([torch.einsum("bd,bdm->bm", fq[:, h], S[:, h // r]) / (fq[:, h] * Z[:, h // r]).sum(-1, keepdim=True)
                              for h in range(q.shape[1])], 1)}


def exact(case, seed):
    return {"gated": _exact_gated, "norm": _exact_norm, "rotary": _exact_rotary, "packed": _exact_packed}[case["op"]](prepare(case, seed))
