"""The compiled allocating calls: what they refuse before a device is touched, that they hold no
references, and calls from several threads at once."""
import gc
import sys
import threading

import pytest
import torch


def calls(la, dev="cpu"):
    """Each call with arguments that are right but for the device, by name."""
    x, w, h = torch.randn(2, 3, 8, device=dev), torch.zeros(8, device=dev), torch.zeros(2, 8, device=dev)
    q, k = torch.randn(2, 3, 2, 8, device=dev), torch.randn(2, 3, 1, 8, device=dev)
    turns = torch.arange(4, device=dev)
    S, Z, one = torch.randn(2, 1, 32, 64, device=dev), torch.ones(2, 1, 32, device=dev), torch.randn(2, 2, 32, device=dev)
    codes, kept = torch.zeros(2, 1, 32, 64, dtype=torch.int8, device=dev), torch.zeros(16, device=dev)
    stat = torch.zeros(2, 3, 2, device=dev)
    return {
        "gated_fwd": (x, x, x, w, h),
        "gated_bwd": (x, x, x, w, kept, x),
        "gated_step": (x[:, 0], x[:, 0], x[:, 0], w, h),
        "norm_fwd": (x, w, w, x, 2),
        "norm_bwd": (x, w, stat, stat, x, x, 2),
        "rotary_fwd": (q, k, turns),
        "rotary_bwd": (q, k, turns),
        "state_pack": (S,),
        "state_unpack": (codes, Z),
        "cross_step_packed": (one, codes, Z, Z),
    }


NAMES = sorted(calls(None))


@pytest.mark.parametrize("name", NAMES)
def test_tensors_only(linattn, name):
    """Anything else in a tensor's place is named; all right, the call asks for a device."""
    args, f = calls(linattn)[name], getattr(linattn, name)
    with pytest.raises(ValueError, match="CUDA device"):
        f(*args)
    for i, t in enumerate(args):
        if not isinstance(t, torch.Tensor):
            continue
        for other in (7, "x", [1.0], t.numpy()):
            with pytest.raises(TypeError, match="a tensor is needed"):
                f(*args[:i], other, *args[i + 1:])


@pytest.mark.parametrize("name", NAMES)
def test_other_device(linattn, name):
    """A tensor on another device than the first's is refused by name."""
    args, f = calls(linattn)[name], getattr(linattn, name)
    for i in range(1, len(args)):
        if isinstance(args[i], torch.Tensor):
            with pytest.raises(ValueError, match="on meta, the call is on cpu"):
                f(*args[:i], args[i].to("meta"), *args[i + 1:])


@pytest.mark.parametrize("name", NAMES)
def test_holds_nothing(linattn, name):
    args, f = calls(linattn)[name], getattr(linattn, name)
    tensors = [t for t in args if isinstance(t, torch.Tensor)]
    before = [sys.getrefcount(t) for t in tensors]
    for _ in range(50):
        with pytest.raises(ValueError):
            f(*args)
    assert [sys.getrefcount(t) for t in tensors] == before


def test_numbers(linattn):
    x, w = torch.zeros(2, 3, 8), torch.zeros(8)
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(ValueError, match="scale"):
            linattn.gated_fwd(x, x, x, w, scale=scale)
    with pytest.raises(TypeError):
        linattn.gated_fwd(x, x, x, w, scale="8")
    with pytest.raises(TypeError):
        linattn.norm_fwd(x, w, groups=2.0)
    with pytest.raises(TypeError):
        linattn.norm_fwd(x, w, eps=None)
    for groups in (0, -1, 3, 1 << 40):
        with pytest.raises(ValueError, match="does not divide 8 columns"):
            linattn.norm_fwd(x, w, groups=groups)
    with pytest.raises(OverflowError):
        linattn.norm_fwd(x, w, groups=1 << 80)


def test_sizes_beyond_the_interface(linattn):
    """Views of one element with more rows than 32 bits count."""
    n = (1 << 31) + 5
    one = torch.zeros(1)
    rows, streams = one.expand(1, n, 1), one.expand(n, 1)
    with pytest.raises(ValueError, match="sizes above"):
        linattn.gated_fwd(rows, rows, rows, one)
    with pytest.raises(ValueError, match="sizes above"):
        linattn.gated_step(streams, streams, streams, one, streams)
    with pytest.raises(ValueError, match="sizes above"):
        linattn.norm_fwd(rows, one)
    q = one.expand(1, n, 1, 2)
    with pytest.raises(ValueError, match="sizes above"):
        linattn.rotary_fwd(q, None, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="sizes above"):
        linattn.state_pack(one.expand(n, 1, 1, 1))
    with pytest.raises(ValueError, match="elements apart"):
        linattn.norm_fwd(torch.as_strided(torch.empty(1), (2, 0), (1 << 31, 1)), torch.zeros(0))


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_releases_everything(cuda, linattn, name):
    """Many calls leave the inputs' references and the device's memory as they were."""
    args = list(calls(linattn, cuda)[name])
    f = getattr(linattn, name)
    if name == "gated_bwd":
        args[4] = linattn.gated_fwd(*args[:4], keep=True)[1]
    tensors = [t for t in args if isinstance(t, torch.Tensor)]
    f(*args)
    torch.cuda.synchronize()
    gc.collect()  # earlier tests' cycles, which would be freed in between
    before, used = [sys.getrefcount(t) for t in tensors], torch.cuda.memory_allocated()
    for _ in range(200):
        f(*args)
    assert [sys.getrefcount(t) for t in tensors] == before and torch.cuda.memory_allocated() <= used


@pytest.mark.gpu
def test_library_errors_come_through(cuda, linattn):
    """A code of the library is raised as LinAttnError with the entry's name."""
    S = torch.zeros(1, 1, 8, 0, device=cuda)
    with pytest.raises(linattn.LinAttnError, match="la_state_pack") as e:
        linattn.state_pack(S)
    assert e.value.code == linattn.LA_ERR_INVALID_ARG


@pytest.mark.gpu
def test_threads(cuda, linattn):
    """Calls of several threads, each on a stream of its own and with more tiles than run at once, give what one
    thread's calls give."""
    g = torch.Generator().manual_seed(4)
    x = [torch.randn(2, 3000, 640, generator=g).to(cuda) for _ in range(6)]
    w = torch.randn(640, generator=g).to(cuda)
    turns, _ = linattn.rotary_turns(32, device=cuda)

    def work(t):
        y, s, mean, rstd = linattn.norm_fwd(t, w, w, x[0])
        z, kept = linattn.gated_fwd(y, s, t, w, keep=True)
        q, _ = linattn.rotary_fwd(z.view(2, 3000, 20, 32), None, turns)
        return [*linattn.gated_bwd(y, s, t, w, kept, z), *linattn.norm_bwd(s, w, mean, rstd, y), q]

    want = [work(t) for t in x]
    torch.cuda.synchronize()
    got, errors = [None] * len(x), []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i] = work(x[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(x))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    linattn.check_device_status()
