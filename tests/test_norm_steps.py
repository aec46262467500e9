"""The norm's gradients where a thread works on more groups than it holds at once, so that the copies into shared memory are
filled again and the sums over rows run over several steps: every way of holding a group, against 64 bits (around64)."""
import pytest
import torch

import around64
from around64 import rounded
from plain64 import F32, within
from test_norm import inputs

CASES = [  # B, N, C, groups, dtype, pad, lengths, residual; blocks of 256 threads or more: 304 at most, and three (two, one) groups at once
    (1, 2000, 2048, 1, "bf16", 0, [1937], True),      # a block a row of 256 threads: 912 rows a step
    (2, 1500, 640, 1, "f32", 0, [1500, 1201], True),
    (1, 3000, 1024, 16, "bf16", 0, None, True),       # heads of 64 on eight threads: 29184 of 48000 a step
    (1, 4000, 1000, 1, "bf16", 8, None, False),       # 128 threads
    (1, 8000, 256, 1, "f32", 4, [7777], False),       # 64 threads
    (1, 16000, 256, 1, "bf16", 0, None, False),       # a warp a row
    (1, 9000, 128, 8, "f32", 0, None, True),          # heads of 16 on four threads
    (1, 1500, 4096, 1, "bf16", 0, None, True),        # two vectors a thread, two rows at once
    (1, 500, 8192, 1, "bf16", 0, [471], True),        # 512 threads, one row at once
    (1, 500, 4100, 1, "f32", 0, None, True),          # four vectors a thread
    (1, 2100, 333, 1, "bf16", 0, None, True),         # value by value: 256 threads
    (1, 12000, 27, 1, "bf16", 3, [11000], True),      # a warp a row
    (2, 9000, 21, 3, "bf16", 0, None, False),         # heads of 7 on eight threads
    (1, 6000, 99, 1, "f32", 0, None, True),           # four values a thread
    (1, 800, 2047, 1, "bf16", 0, None, True),         # eight values a thread
    (1, 400, 8191, 1, "bf16", 0, None, False),        # 1024 threads
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,C,G,dtype,pad,lengths,residual", CASES)
def test_gradients_over_several_steps(cuda, linattn, B, N, C, G, dtype, pad, lengths, residual):
    x, w, b, res, dy, ds = inputs(B, N, C, dtype, pad, C)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=cuda)
    res, ds = (res[..., :C], ds) if residual else (None, None)
    dev = lambda t: None if t is None else t.to(cuda)  # noqa: E731
    y, s, mean, rstd = linattn.norm_fwd(dev(x)[..., :C], dev(w), dev(b), residual=dev(res), groups=G, lengths=n)
    dx, dw, db = linattn.norm_bwd(s, dev(w), mean, rstd, dev(dy), dev(ds), groups=G, lengths=n)
    want = around64.norm(x[..., :C], w, b, res, G, 1e-5, lengths, dy, ds)
    # sums over rows: not a half step a row but one for each of a chain's additions: at most 16 of a thread's groups, 64 of a
    # block's groups, 110 of every 32nd partial sum and 32
    live = torch.arange(N)[None, :] < torch.tensor([N] * B if lengths is None else lengths)[:, None]
    d = torch.where(live[..., None], dy.double(), 0.0)
    xh = ((want["s"][0].unflatten(-1, (G, -1)) - want["mean"][0].unflatten(-1, (G, 1))) * want["rstd"][0].unflatten(-1, (G, 1))).flatten(2)
    for name, terms in (("dw", d * xh), ("db", d)):
        value, bound = want[name]
        want[name] = value, bound + (16 + 64 + 110 + 32 - (B * N + 16)) * F32 * terms.abs().sum((0, 1))
    for name, t in zip(("y", "dx", "dw", "db"), (y, dx, dw, db)):
        within(t, want[name][0], rounded(*want[name], dtype), name)
