"""The compiled allocating calls: what they refuse before a device is touched, that they hold no
references, and calls from several threads at once."""
import gc
import os
import subprocess
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


def around(la, x, w, turns, h, Z):
    """Every kind of call behind x, a tensor that another stream writes."""
    y, s, mean, rstd = la.norm_fwd(x, w, w, x)
    z, kept = la.gated_fwd(x, y, s, w, keep=True)
    state = h.clone()
    codes, scale = la.state_pack(x[:, :64, :64].reshape(2, 1, 64, 64).contiguous())
    q = x[:, 0].reshape(2, 10, 64).contiguous()
    return [y, *la.norm_bwd(x, w, mean, rstd, y), z, *la.gated_bwd(x, y, s, w, kept, x), la.gated_step(x[:, 1], y[:, 1], s[:, 1], w, state), state,
            la.rotary_fwd(x.view(2, 300, 10, 64), None, turns)[0], la.state_unpack(codes, scale), la.cross_step_packed(q, codes, scale, Z)]


def late(x, y):
    """y into x at the end of some hundred microseconds of work."""
    t = torch.randn(2048, 2048, device=x.device)
    for _ in range(20):
        t = t @ t * 1e-3
    x.copy_(y + 0 * t.nan_to_num().clamp(-1, 1)[0, 0])


@pytest.fixture(scope="module")
def behind(cuda, linattn):
    g = torch.Generator().manual_seed(6)
    y = [torch.randn(2, 300, 640, generator=g).to(cuda) for _ in range(3)]
    turns, _ = linattn.rotary_turns(32, device=cuda)
    rest = torch.randn(640, generator=g).to(cuda), turns, torch.randn(2, 640, generator=g).to(cuda), torch.rand(2, 1, 64, generator=g).to(cuda)
    want = [around(linattn, t, *rest) for t in y]
    torch.cuda.synchronize()
    return y, rest, want


@pytest.mark.gpu
def test_behind_another_stream(cuda, linattn, behind):
    """Calls that wait for another stream's event read what it wrote, not what was there."""
    y, rest, want = behind
    x, side = torch.zeros_like(y[0]), torch.cuda.Stream()
    for t, expect in zip(y, want):
        for first in range(5):
            x.zero_()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                late(x, t)
            linattn.norm_fwd(y[0], rest[0])  # a kernel of the same stream just before the wait
            torch.cuda.current_stream().wait_stream(side)
            calls_ = [lambda: linattn.rotary_fwd(x.view(2, 300, 10, 64), None, rest[1])[0], lambda: linattn.norm_fwd(x, rest[0], rest[0], x)[0],
                      lambda: linattn.gated_fwd(x, x, x, rest[0]), lambda: linattn.gated_step(x[:, 1], x[:, 1], x[:, 1], rest[0], rest[2].clone()),
                      lambda: linattn.state_pack(x.view(1, 375, 16, 64))[0]]
            got = calls_[first]()  # each as the first behind the wait
            rest_of = around(linattn, x, *rest)
            torch.cuda.synchronize()
            assert torch.equal(got, calls_[first]())
            assert all(torch.equal(a, b) for a, b in zip(rest_of, expect))


@pytest.mark.gpu
def test_captured_behind_another_stream(cuda, linattn, behind):
    """The same in a graph that forks and joins."""
    y, rest, want = behind
    x, source, side, main = torch.zeros_like(y[0]), y[0].clone(), torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        late(x, source)
        around(linattn, x, *rest)
    main.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            late(x, source)
        linattn.norm_fwd(y[0], rest[0])
        main.wait_stream(side)
        got = around(linattn, x, *rest)
    for _ in range(3):
        for t, expect in zip(y, want):
            x.zero_()
            source.copy_(t)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, expect))
    linattn.check_device_status()


FIRST = """
import torch
import kernelized_causal_attention_gb300 as la
g = torch.Generator().manual_seed(1)
x, w = torch.randn(2, 300, 640, generator=g).cuda(), torch.randn(640, generator=g).cuda()
def run():
    y, s, mean, rstd = la.norm_fwd(x, w, w)
    z, kept = la.gated_fwd(x, y, x, w, keep=True)
    return [y, z, *la.gated_bwd(x, y, x, w, kept, x), *la.norm_bwd(x, w, mean, rstd, y)]
graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(graph, stream=s):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
la.check_device_status()
"""


@pytest.mark.gpu
def test_first_call_is_captured(cuda, linattn):
    """A process whose first calls are captured."""
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr
