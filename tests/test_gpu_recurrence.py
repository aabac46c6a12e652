"""GPU parity of the gated linear recurrence (gs_recurrence_fwd / _bwd)
against the float64 oracle (oracle/training.py), element by element within
the bound of float32 arithmetic that the oracle derives with each value (an
error can only come from roundings on the element's own chain).
"""
import sys

import numpy as np
import pytest

from gpu_helpers import to_np
from oracle import training as tr

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def _torch_type(dtype):
    import torch
    return dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[dtype]


def _inputs(seed, B, T, D, dtype, sigmoid, ragged=False, restarts=False, remember=2.0):
    """Host inputs rounded to dtype (as float64 arrays) and the device tensors that hold them."""
    import torch
    rng = np.random.default_rng(seed)
    gate = rng.normal(remember, 2.0, (B, T, D))
    if not sigmoid:
        gate = 1.0 / (1.0 + np.exp(-gate))
    t = _torch_type(dtype)
    dev = {k: torch.from_numpy(a).to(t).cuda() for k, a in
           dict(gate=gate, x=rng.normal(0, 1, (B, T, D)), grad_h=rng.normal(0, 1, (B, T, D))).items()}
    host = {k: to_np(a.double()) for k, a in dev.items()}
    for k in ("h0", "grad_last"):
        host[k] = rng.normal(0, 1, (B, D)).astype(np.float32)
        dev[k] = torch.from_numpy(host[k]).cuda()
    host["lengths"] = host["restart"] = dev["lengths"] = dev["restart"] = None
    if ragged:
        n = rng.integers(0, T + 1, B).astype(np.int32)
        n[:3] = [T, 0, min(1, T)][:min(B, 3)]
        host["lengths"], dev["lengths"] = n, torch.from_numpy(n).cuda()
    if restarts:
        z = (rng.random((B, T)) < 5.0 / (T + 5)).astype(np.uint8)
        host["restart"], dev["restart"] = z, torch.from_numpy(z).cuda()
    return host, dev


def _oracle(host, dtype, sigmoid, back=True):
    return tr.recurrence(host["gate"], host["x"], host["h0"], sigmoid, host["lengths"], host["restart"],
                         host["grad_h"] if back else None, host["grad_last"] if back else None, dtype)


def _run(dev, sigmoid, back=True):
    import torch
    import gaussian_splatting_tile_amd as gs
    kw = dict(gating=gs.GATE_SIGMOID if sigmoid else gs.GATE_LINEAR, lengths=dev["lengths"], restart=dev["restart"])
    out = gs.recurrence_fwd(dev["gate"], dev["x"], h0=dev["h0"], checkpoints=back, **kw)
    if back:
        out.update(gs.recurrence_bwd(dev["gate"], dev["x"], dev["grad_h"], h0=dev["h0"], ckpt=out["ckpt"],
                                     grad_last=dev["grad_last"], **kw))
    torch.cuda.synchronize()
    return out


def _check(out, ref, what):
    for k, (value, bound) in ref.items():
        got = to_np(out[k].double())
        off = np.abs(got - value)
        bad = ~(off <= bound)
        assert not bad.any(), (what, k, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], value[bad][:3],
                               bound[bad][:3])


SHAPES = [(1, 1, 1), (3, 1, 130), (2, 2, 63), (3, 3, 140), (2, 4, 66), (4, 5, 64), (1, 15, 64), (2, 16, 65), (3, 17, 128), (2, 31, 3), (2, 33, 200),
          (1, 64, 257), (2, 65, 66), (3, 127, 70), (3, 128, 64), (4, 129, 37), (1, 255, 130), (4, 300, 96), (2, 1025, 5),
          (1, 4609, 3), (5, 777, 129)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_recurrence_parity(dtype, sigmoid, B, T, D):
    for ragged, restarts in ((False, False), (True, True)):
        say(f"[recurrence {B}x{T}x{D} {dtype} sigmoid={sigmoid} ragged={ragged}]")
        host, dev = _inputs(B * 7919 + T * 31 + D, B, T, D, dtype, sigmoid, ragged, restarts)
        _check(_run(dev, sigmoid), _oracle(host, dtype, sigmoid), (ragged, restarts))


@pytest.mark.parametrize("B,T,D", [(0, 4, 8), (3, 4, 0), (3, 0, 8)])
def test_recurrence_of_nothing(B, T, D):
    import torch
    import gaussian_splatting_tile_amd as gs
    say(f"[recurrence of nothing {B}x{T}x{D}]")
    z = torch.zeros((B, T, D), device="cuda")
    h0, gl = torch.randn((B, D), device="cuda"), torch.randn((B, D), device="cuda")
    out = gs.recurrence_fwd(z, z, h0=h0, checkpoints=True)
    back = gs.recurrence_bwd(z, z, z, h0=h0, ckpt=out["ckpt"], grad_last=gl)
    torch.cuda.synchronize()
    if T == 0:  # the state passes through
        assert torch.equal(out["h_last"], h0) and torch.equal(back["grad_h0"], gl)


def test_recurrence_without_optional_arguments():
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[recurrence without h0, grad_last]")
    host, dev = _inputs(11, 2, 300, 40, "f32", True)
    out = gs.recurrence_fwd(dev["gate"], dev["x"], gating=gs.GATE_SIGMOID, checkpoints=True)
    back = gs.recurrence_bwd(dev["gate"], dev["x"], dev["grad_h"], ckpt=out["ckpt"], gating=gs.GATE_SIGMOID)
    torch.cuda.synchronize()
    ref = tr.recurrence(host["gate"], host["x"], None, True, grad_h=host["grad_h"])
    _check(dict(out, **back), ref, "no h0")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 130, 131])
def test_recurrence_strided_inputs(dtype, D):
    """gate and x as halves of one projection, one of them odd in its first element, and a gate
    that is the same at every step (stride 0)."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say(f"[recurrence strided {dtype} D={D}]")
    B, T = 2, 200
    host, dev = _inputs(D, B, T, D, dtype, False)
    both = torch.empty((B, T + 3, 2 * D + 1), dtype=_torch_type(dtype), device="cuda")
    both[:, :T, 1:D + 1], both[:, :T, D + 1:] = dev["gate"], dev["x"]
    d2 = dict(dev, gate=both[:, :T, 1:D + 1], x=both[:, :T, D + 1:])
    ref = _oracle(host, dtype, False)
    _check(_run(d2, False), ref, "halves")
    same = dev["gate"][:, :1].expand(B, T, D)
    h2 = dict(host, gate=np.repeat(host["gate"][:, :1], T, 1))
    _check(_run(dict(dev, gate=same), False), _oracle(h2, dtype, False), "one gate")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T", [20, 128, 300])
def test_recurrence_padding_is_not_read(sigmoid, T):
    """NaN and infinities behind the lengths and in dropped states leave no trace."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say(f"[recurrence padding T={T} sigmoid={sigmoid}]")
    B, D = 6, 70
    host, dev = _inputs(T, B, T, D, "f32", sigmoid, ragged=True, restarts=True)
    ref = _oracle(host, "f32", sigmoid)
    for k, v in (("gate", float("nan")), ("x", float("inf")), ("grad_h", float("nan"))):
        dev[k] = dev[k].clone()
        for b, n in enumerate(host["lengths"]):
            dev[k][b, n:] = v
    _check(_run(dev, sigmoid), ref, "padding")
    # a state that is not finite ends at a restart
    dev["restart"], host["restart"] = dev["restart"].clone(), host["restart"].copy()
    dev["restart"][0, T // 2] = 1
    host["restart"][0, T // 2] = 1
    for bad in (float("nan"), float("inf")):
        dev["h0"] = dev["h0"].clone()
        dev["h0"][0] = bad
        h0 = host["h0"].copy()
        h0[0] = 0.0
        out = _run(dev, sigmoid, back=False)
        want = _oracle(dict(host, h0=h0), "f32", sigmoid, back=False)
        got, (value, bound) = to_np(out["h"].double()), want["h"]
        assert (np.abs(got[0, T // 2:] - value[0, T // 2:]) <= bound[0, T // 2:]).all(), bad
        first = int(np.argmax(host["restart"][0] != 0))
        assert not np.isfinite(got[0, :first]).any()


def test_recurrence_non_finite_values_stay():
    """A NaN gate, and an infinite input, reach every later state of their channel and no other channel."""
    import torch
    say("[recurrence non-finite]")
    host, dev = _inputs(3, 1, 400, 96, "f32", False)
    dev["gate"][0, 50, 7] = float("nan")
    dev["x"][0, 60, 9] = float("inf")
    got = to_np(_run(dev, False, back=False)["h"])
    assert np.isnan(got[0, 50:, 7]).all() and not np.isfinite(got[0, 60:, 9]).any()
    assert np.isfinite(got[0, :50, 7]).all() and np.isfinite(got[0, :60, 9]).all()
    other = np.ones(96, bool)
    other[[7, 9]] = False
    assert np.isfinite(got[0][:, other]).all()


@pytest.mark.parametrize("gate", [0.0, 1.0, -1.0, 1e-30])
def test_recurrence_edge_gates(gate):
    """Gates of 0, +-1 and ones whose product over a chunk underflows; states of 0 in front."""
    import torch
    say(f"[recurrence gate {gate}]")
    host, dev = _inputs(4, 2, 500, 33, "f32", False)
    dev["gate"].fill_(gate)
    host["gate"] = to_np(dev["gate"].double())
    _check(_run(dev, False), _oracle(host, "f32", False), gate)


def test_recurrence_growing_gates_with_a_zero_state():
    """Gates of 2: the product over 128 steps overflows float32, but a state that stays 0 stays 0."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[recurrence gates of 2]")
    gate, x = torch.full((1, 600, 65), 2.0, device="cuda"), torch.zeros((1, 600, 65), device="cuda")
    out = gs.recurrence_fwd(gate, x)
    torch.cuda.synchronize()
    assert not out["h"].any() and not out["h_last"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_recurrence_step_by_step_equals_the_whole(dtype):
    """T = 1 calls that keep their state in one buffer give what one call over all steps gives,
    within twice the bound (both differ from the exact states by at most it)."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say(f"[recurrence steps {dtype}]")
    host, dev = _inputs(21, 3, 40, 100, dtype, True)
    whole = _run(dev, True, back=False)
    state = dev["h0"].clone()
    ref = _oracle(host, dtype, True, back=False)
    for t in range(40):
        out = gs.recurrence_fwd(dev["gate"][:, t:t + 1], dev["x"][:, t:t + 1], h0=state, gating=gs.GATE_SIGMOID,
                                out=dict(h_last=state))
        assert out["h_last"] is state
        off = (out["h"][:, 0].double() - whole["h"][:, t].double()).abs().cpu().numpy()
        assert (off <= 2 * ref["h"][1][:, t]).all(), t
    assert ((state - whole["h_last"]).abs().cpu().numpy() <= 2 * ref["h_last"][1]).all()


@pytest.mark.parametrize("T", [100, 1000])
def test_recurrence_state_in_place_over_many_steps(T):
    """h_last may be h0 at any length."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say(f"[recurrence in place T={T}]")
    host, dev = _inputs(T, 2, T, 70, "f32", False)
    a = gs.recurrence_fwd(dev["gate"], dev["x"], h0=dev["h0"])
    state = dev["h0"].clone()
    b = gs.recurrence_fwd(dev["gate"], dev["x"], h0=state, out=dict(h_last=state))
    torch.cuda.synchronize()
    assert torch.equal(a["h"], b["h"]) and torch.equal(a["h_last"], state)


def test_recurrence_is_deterministic_and_uses_its_stream():
    import torch
    say("[recurrence deterministic]")
    host, dev = _inputs(5, 2, 6000, 200, "bf16", True, ragged=True, restarts=True)
    first = _run(dev, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            again = _run(dev, True)
        for k in ("h", "h_last", "grad_gate", "grad_x", "grad_h0"):
            assert torch.equal(first[k], again[k]), k
        n = [int(v) for v in host["lengths"]]
        for b, length in enumerate(n):  # rows behind the length are not written
            rows = max(0, -(-length // 128) - 1)
            assert torch.equal(first["ckpt"][b, :rows], again["ckpt"][b, :rows])


@pytest.mark.parametrize("dtype,D", [("f32", 70), ("bf16", 130), ("f16", 33)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T", [300, 128 * 67 + 5])
def test_recurrence_without_waiting_gives_the_same_bits(monkeypatch, dtype, D, sigmoid, T):
    """A chunk that finds nothing of what the chunks before it publish computes it from the
    inputs: forced for every chunk, over more than one group of groups, it changes no bit."""
    say(f"[recurrence alone {dtype} D={D} T={T} sigmoid={sigmoid}]")
    host, dev = _inputs(T + D, 2, T, D, dtype, sigmoid, ragged=False, restarts=T == 300, remember=4.0)
    keys = ("h", "h_last", "grad_gate", "grad_x", "grad_h0", "ckpt")
    want = _run(dev, sigmoid)
    monkeypatch.setenv("GS_RECURRENCE_PATIENCE", "0")
    got = _run(dev, sigmoid)
    for k in keys:
        assert (want[k] == got[k]).all(), k


def test_recurrence_in_a_graph():
    """Recorded once and replayed on changing inputs, with eager work between the replays."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[recurrence graph]")
    host, dev = _inputs(6, 2, 700, 90, "f32", False, restarts=True)
    out = {}
    kw = dict(restart=dev["restart"])

    def call():
        f = gs.recurrence_fwd(dev["gate"], dev["x"], h0=dev["h0"], checkpoints=True, **kw)
        b = gs.recurrence_bwd(dev["gate"], dev["x"], dev["grad_h"], h0=dev["h0"], ckpt=f["ckpt"],
                              grad_last=dev["grad_last"], **kw)
        return dict(f, **b)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for k in range(4):
        dev["x"].copy_(torch.randn_like(dev["x"]))
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        torch.cuda.synchronize()
        for name in ("h", "h_last", "grad_gate", "grad_x", "grad_h0"):
            assert torch.equal(out[name], want[name]), (k, name)


def test_recurrence_gradients_match_differences():
    """Central differences of the kernel's own forward in float32. With a step of 2^-6 and a
    loss that is a sum of products of at most one varied gate each (the recurrence is linear in
    each input and in each single gate) a difference has no truncation error: only the loss's
    rounding, bounded by the states' error bounds, over twice the step."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[recurrence differences]")
    B, T, D, d = 1, 140, 4, 2.0 ** -6
    host, dev = _inputs(8, B, T, D, "f32", False)
    g = host["grad_h"]

    def loss(**kw):
        a = dict(dev, **kw)
        out = gs.recurrence_fwd(a["gate"], a["x"], h0=a["h0"])
        return float((to_np(out["h"].double()) * g).sum() + (to_np(out["h_last"].double()) * host["grad_last"]).sum())

    out = _run(dev, False)
    ref = _oracle(host, "f32", False)
    slack = (np.abs(g) * ref["h"][1]).sum() + (np.abs(host["grad_last"]) * ref["h_last"][1]).sum()
    for name, grad in (("gate", "grad_gate"), ("x", "grad_x")):
        for t in (0, 1, 63, 127, 128, 139):
            lo, hi = dev[name].clone(), dev[name].clone()
            lo[0, t, 2] -= d
            hi[0, t, 2] += d
            width = float(hi[0, t, 2].double() - lo[0, t, 2].double())
            num = (loss(**{name: hi}) - loss(**{name: lo})) / width
            # varied gates stay below 1 + d, so states grow by at most that factor once: twice the slack covers both
            assert abs(num - float(out[grad][0, t, 2])) <= 4 * slack / width, (name, t)


def test_recurrence_long_sequence():
    """65,536 steps: against the oracle on few channels, offsets far into the sequence."""
    say("[recurrence 65536 steps]")
    host, dev = _inputs(9, 1, 65536, 8, "f32", False, restarts=True, remember=6.0)
    _check(_run(dev, False), _oracle(host, "f32", False), "long")


def test_recurrence_offsets_past_32_bits():
    """Element offsets past 2^31 (bf16, 2.2e9 elements in h): the last channels' states."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[recurrence 2.2e9 elements]")
    T, D = 17, 1 << 27
    t = torch.bfloat16
    gate = torch.full((1, 1, 1), 0.5, dtype=t, device="cuda").expand(1, T, D)
    if gate.stride(2) != 1:
        gate = torch.full((1, 1, D), 0.5, dtype=t, device="cuda").expand(1, T, D)
    x = torch.arange(D, device="cuda").remainder_(97).to(t)[None, None].expand(1, T, D)
    out = gs.recurrence_fwd(gate, x)
    torch.cuda.synchronize()
    # h_t = x (2 - 2^-t): x below 97 has 7 bits and t <= 16, so float32 holds every state exactly
    last = (x[0, 0].float() * (2.0 - 2.0 ** -(T - 1)))
    assert torch.equal(out["h_last"][0], last)
    assert torch.equal(out["h"][0, T - 1], last.to(t))


def test_recurrence_refuses():
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[recurrence refusals]")
    x = torch.zeros((2, 200, 8), device="cuda")
    with pytest.raises(ValueError):
        gs.recurrence_fwd(x, x[:, :100])
    with pytest.raises(ValueError):
        gs.recurrence_fwd(x, x.bfloat16())
    with pytest.raises(TypeError):
        gs.recurrence_fwd(x.double(), x.double())
    with pytest.raises(TypeError):
        gs.recurrence_fwd(x.cpu(), x.cpu())
    with pytest.raises(ValueError):
        gs.recurrence_fwd(x.transpose(1, 2), x.transpose(1, 2))
    with pytest.raises(ValueError):
        gs.recurrence_fwd(x, x, h0=torch.zeros((2, 9), device="cuda"))
    with pytest.raises(TypeError):
        gs.recurrence_fwd(x, x, lengths=torch.zeros((2,), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        gs.recurrence_fwd(x, x, restart=torch.zeros((2, 8), dtype=torch.uint8, device="cuda"))
    with pytest.raises(gs.GsError):
        gs.recurrence_fwd(x, x, gating=2)
    with pytest.raises(gs.GsError):
        gs.recurrence_bwd(x, x, x)  # 200 steps need the checkpoints
    with pytest.raises(gs.GsError):  # 200 steps need a workspace of some size
        gs.recurrence_fwd(x, x, scratch=torch.empty((8,), dtype=torch.uint8, device="cuda"))
