"""GPU tests of the sequence and training calls on a stream that is not the current one: what
a call allocates is ordered with its own stream, and what it returns with the caller's."""
import sys

import pytest

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def _busy(big):
    """Some 10 ms of work on the current stream."""
    for _ in range(40):
        big.mul_(1.0)


def _calls(kind, seed):
    """A call with `stream` on fresh inputs: {name: tensor} of what it allocates."""
    import torch
    import gaussian_splatting_tile_amd as gs
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    grads = [torch.randn(100_000, generator=g, device="cuda"), torch.randn(77, generator=g, device="cuda")]
    x = torch.randn((1, 700, 128), generator=g, device="cuda")
    if kind == "norm":
        return lambda stream: dict(norm=gs.grad_norm(grads, stream=stream))
    if kind == "clip":
        out = [torch.empty_like(t) for t in grads]
        return lambda stream: dict(norm=gs.clip_grads(grads, 1.0, out=out, stream=stream))
    if kind == "list":
        lst = gs.GradList(grads)
        return lambda stream: dict(norm=lst.norm(stream=stream))
    if kind == "fwd":
        return lambda stream: gs.recurrence_fwd(x, x, gating=gs.GATE_SIGMOID, checkpoints=True, stream=stream)
    f = gs.recurrence_fwd(x, x, gating=gs.GATE_SIGMOID, checkpoints=True)
    return lambda stream: gs.recurrence_bwd(x, x, x, ckpt=f["ckpt"], gating=gs.GATE_SIGMOID, stream=stream)


KINDS = ["norm", "clip", "list", "fwd", "bwd"]


@pytest.mark.parametrize("kind", KINDS)
def test_memory_of_pending_work_is_not_taken(kind):
    """The current stream still has a write to memory that is free for its own next allocation: a
    call on another stream does not wait for it, so none of its tensors may lie there."""
    import torch
    say(f"[stream, pending work, {kind}]")
    big = torch.ones(1 << 27, device="cuda")
    call, side = _calls(kind, 1), torch.cuda.Stream()
    want = {k: t.clone() for k, t in call(None).items()}
    torch.cuda.synchronize()
    for _ in range(3):
        free = [torch.empty_like(t) for t in want.values()] + [torch.empty(1 << 16, dtype=torch.uint8, device="cuda")]
        _busy(big)
        for t in free:
            t.fill_(7)
        del free, t
        got = call(side)
        torch.cuda.synchronize()
        for k, t in got.items():
            assert torch.equal(t, want[k]), k


@pytest.mark.parametrize("kind", KINDS)
def test_results_may_be_used_and_dropped_on_the_callers_stream(kind):
    """A result read on the current stream (behind the side stream) and dropped before that
    read has run is not written over by the next call on the side stream."""
    import torch
    say(f"[stream, dropped results, {kind}]")
    big = torch.ones(1 << 27, device="cuda")
    first, second, side = _calls(kind, 1), _calls(kind, 2), torch.cuda.Stream()
    want = {k: t.clone() for k, t in first(None).items()}
    torch.cuda.synchronize()
    for _ in range(3):
        got = first(side)
        torch.cuda.current_stream().wait_stream(side)
        _busy(big)
        read = {k: t.clone() for k, t in got.items()}
        del got
        second(side)
        second(side)
        torch.cuda.synchronize()
        for k, t in read.items():
            assert torch.equal(t, want[k]), k


def test_objects_may_be_dropped_behind_their_calls():
    """A GradList and an Adam made on the current stream, used on another behind long work
    there, and dropped at once: what the current stream allocates next does not lie in them."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[stream, dropped objects]")
    big = torch.ones(1 << 27, device="cuda")
    n = 300_000
    g = torch.randn(n, device="cuda")
    p = torch.ones(n, device="cuda")
    q = p.clone()
    gs.Adam([q], [g], lr=0.01, max_norm=1.0).step()
    out = torch.empty_like(g)
    want = gs.clip_grads([g], 1.0, out=[out])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (True, False):
        p.fill_(1.0)
        clipped, norm = torch.empty_like(g), torch.zeros((), device="cuda")
        lst, adam = gs.GradList([g], out=[clipped]), gs.Adam([p], [g], lr=0.01, max_norm=1.0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _busy(big)
            if not given:
                lst.clip(1.0, out=norm)
                adam.step()
        if given:
            lst.clip(1.0, out=norm, stream=side)
            adam.step(stream=side)
        del lst, adam
        for _ in range(4):  # the sizes of the moments, the workspace and the scalars
            for shape, dtype in (((n,), torch.float32), ((1 << 14,), torch.uint8), ((1,), torch.int64)):
                torch.full(shape, 7, dtype=dtype, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(p, q) and torch.equal(clipped, out) and torch.equal(norm, want)


def test_calls_make_their_device_current(monkeypatch):
    """Where another device than the tensors' is current, the launch runs with theirs."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[device of a call]")
    x = torch.randn((2, 300, 64), device="cuda")
    want = gs.recurrence_fwd(x, x, gating=gs.GATE_SIGMOID, checkpoints=True)
    norm = gs.grad_norm([x])
    entered, real = [], torch.cuda.device.__enter__
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch.cuda.device, "__enter__", lambda self: (entered.append(self.idx), real(self))[1])
    got = gs.recurrence_fwd(x, x, gating=gs.GATE_SIGMOID, checkpoints=True)
    assert entered == [x.device.index]
    back = gs.recurrence_bwd(x, x, x, ckpt=got["ckpt"], gating=gs.GATE_SIGMOID)
    p = torch.ones_like(x)
    adam = gs.Adam([p], [back["grad_x"]], max_norm=1.0)
    again = gs.grad_norm([x])
    adam.step()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert entered == [x.device.index] * 4
    assert torch.equal(got["h"], want["h"]) and torch.equal(again, norm) and int(adam.steps) == 1
