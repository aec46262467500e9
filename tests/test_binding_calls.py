"""How the calls of the layer with a data-dependent decay may be written: by keyword."""
import inspect

import pytest
import torch

CALLS = ("short_conv_fwd", "short_conv_bwd", "short_conv_step", "scan_fwd", "scan_bwd", "scan_step", "cross_fwd", "cross_bwd", "cross_step")


def cpu_arguments():
    z = torch.zeros
    x, dt, A, b = z(2, 5, 4, 16), z(2, 5, 4), z(4), z(2, 5, 1, 16)
    scan = dict(x=x, dt=dt, A=A, Bm=b, Cm=b, skip=None, dt_bias=None)
    step = {n: t[:, 0] if t is not None and t.dim() > 1 else t for n, t in scan.items()}
    conv = dict(x=z(2, 5, 8), w=z(8, 4), bias=None)
    q, k, v, S, Z = z(1, 2, 5, 16), z(1, 1, 7, 16), z(1, 1, 7, 32), z(1, 1, 16, 32), z(1, 1, 16)
    cross = dict(q=q, k=k, v=v, lengths=None)
    return {
        "short_conv_fwd": conv, "short_conv_bwd": dict(conv, dy=z(2, 5, 8)), "short_conv_step": dict(conv, x=z(2, 8), state=z(2, 3, 8)),
        "scan_fwd": scan, "scan_bwd": dict(scan, dy=x), "scan_step": dict(step, S=z(2, 4, 16, 16)),
        "cross_fwd": cross, "cross_bwd": dict(cross, out=z(1, 2, 5, 32), den=z(1, 2, 5), S=S, Z=Z, dout=z(1, 2, 5, 32)),
        "cross_step": dict(q=z(1, 2, 16), S=S, Z=Z),
    }


@pytest.mark.parametrize("name", CALLS)
def test_by_keyword(linattn, name):
    """Every argument by its documented name: the call gets as far as asking for a CUDA device."""
    f, kw = getattr(linattn, name), cpu_arguments()[name]
    assert set(kw) <= set(inspect.signature(f).parameters)
    with pytest.raises(ValueError, match="CUDA device"):
        f(**kw)
    first = next(iter(kw))
    with pytest.raises(TypeError, match=first):
        f(**{n: t for n, t in kw.items() if n != first})
