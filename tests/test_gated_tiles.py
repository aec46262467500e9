"""The gated recurrence where a resident block works on several tiles, and where a NaN goes, against 64 bits (around64)."""
import pytest
import torch

import around64
from around64 import rounded
from plain64 import within
from test_gated import cut, inputs, number

CASES = [  # B, N, C, dtype, pad, lengths: 561 to 864 gradient tiles of 64 rows and channels, on two blocks an SM
    (3, 700, 1030, "f32", 0, [700, 513, 80]),
    (3, 700, 1031, "bf16", 0, [130, 700, 699]),
    (3, 700, 1030, "bf16", 2, None),
    (2, 1100, 1536, "f32", 0, None),
    (2, 1100, 1536, "bf16", 16, [1100, 970]),
    (2, 1100, 1536, "bf16", 0, [0, 1100]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,C,dtype,pad,lengths", CASES)
def test_several_tiles_a_block(cuda, linattn, B, N, C, dtype, pad, lengths):
    wide, lam, dy, h = inputs(B, N, C, dtype, pad, 20, -10, -4)
    n, a, hd = number(lengths, cuda), cut(wide, C, cuda), h.to(cuda)
    assert -(-N // 64) * -(-C // 64) * B > 3 * torch.cuda.get_device_properties(cuda).multi_processor_count
    y, kept = linattn.gated_fwd(*a, lam.to(cuda), h=hd, lengths=n, keep=True)
    got = linattn.gated_bwd(*a, lam.to(cuda), kept, dy.to(cuda), lengths=n)
    want = around64.gated(*cut(wide, C), lam, 8.0, h, lengths, dy)
    for name, t in zip(("y", "dx", "dr", "di", "dlam"), (y, *got)):
        within(t, want[name][0], rounded(*want[name], dtype), name)
    within(hd, *want["h"], "state")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", range(5))
def test_a_nan_goes_where_the_formulas_take_it(cuda, linattn, dtype, which):
    """In x, r, i, dy at a row, or in the first state: NaN in the same places of every result as in 64 bits, none elsewhere."""
    wide, lam, dy, h = inputs(2, 200, 32, dtype, 0, 21)
    x, r, i = (t.contiguous() for t in cut(wide, 32))
    args = (x, r, i, dy)
    if which < 4:
        args[which][1, 130, 5] = float("nan")
    else:
        h[1, 5] = float("nan")
    a, hd = [t.to(cuda) for t in (x, r, i, lam)], h.to(cuda)
    y, kept = linattn.gated_fwd(*a, h=hd, keep=True)
    got = linattn.gated_bwd(*a, kept, dy.to(cuda))
    want = around64.gated(x, r, i, lam, 8.0, h, None, dy)
    some = 0
    for name, t in zip(("y", "dx", "dr", "di", "dlam", "h"), (y, *got, hd)):
        bad = torch.isnan(want[name][0])
        assert torch.equal(torch.isnan(t.cpu()), bad), name
        assert torch.isfinite(t.cpu()[~bad]).all(), name
        some += int(bad.sum())
        if bad.dim() == 3:
            assert not bad[0].any() and not bad[..., [c for c in range(32) if c != 5]].any()
    assert some > 0 and bool(torch.isnan(got[3][5]))
