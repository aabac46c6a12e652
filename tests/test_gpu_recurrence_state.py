"""GPU tests of the gated linear recurrence's state across chunks of steps: one buffer for the
state in front and behind, however the chunks get it. Inputs and oracle as in
test_gpu_recurrence.py."""
import numpy as np
import pytest

from gpu_helpers import to_np
from test_gpu_recurrence import _check, _inputs, _oracle, _run, _torch_type, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [("f32", 33), ("f32", 130), ("bf16", 130), ("bf16", 63), ("f16", 64)])
@pytest.mark.parametrize("T", [100, 129, 300, 128 * 67 + 5])
@pytest.mark.parametrize("waiting", [True, False])
def test_state_in_place_without_waiting(monkeypatch, dtype, D, T, waiting):
    """h_last may be h0 at any length: also where chunks compute for themselves what the chunks
    before them have not given yet, and so read the initial state at any later time."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say(f"[recurrence in place {dtype} D={D} T={T} waiting={waiting}]")
    _, dev = _inputs(T + D, 3, T, D, dtype, True, ragged=True, remember=6.0)
    want = _run(dev, True, back=False)
    if not waiting:
        monkeypatch.setenv("GS_RECURRENCE_PATIENCE", "0")
    kw = dict(gating=gs.GATE_SIGMOID, lengths=dev["lengths"])
    for _ in range(3):
        state = dev["h0"].clone()
        got = gs.recurrence_fwd(dev["gate"], dev["x"], h0=state, out=dict(h_last=state), checkpoints=True, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got["h"], want["h"]) and torch.equal(state, want["h_last"])
    if T > 128 and waiting:  # checkpoints of a state in place serve the backward as any
        rows = (T + 127) // 128 - 1
        full = gs.recurrence_fwd(dev["gate"], dev["x"], h0=dev["h0"], checkpoints=True, **kw)["ckpt"]
        n = int(dev["lengths"][0])
        assert n == T and torch.equal(got["ckpt"][0, :rows], full[0, :rows])


def _of_gates(dtype, gate, h0, grad_last, x=None):
    """Inputs with these gates [T, D], both ends of the states' and gradients' chains given."""
    import torch
    T, D = gate.shape
    host, dev = _inputs(T + D, 1, T, D, dtype, False)
    t = _torch_type(dtype)
    dev["gate"] = torch.from_numpy(gate[None]).to(t).cuda()
    dev["x"] = torch.from_numpy(np.zeros((1, T, D)) if x is None else x[None]).to(t).cuda()
    dev["grad_h"] = torch.zeros((1, T, D), dtype=t, device="cuda")
    for k in ("gate", "x", "grad_h"):
        host[k] = to_np(dev[k].double())
    for k, v in (("h0", h0), ("grad_last", grad_last)):
        host[k] = np.full((1, D), v, np.float32)
        dev[k] = torch.from_numpy(host[k]).cuda()
    return host, dev


# The oracle's bounds are relative. Where a gradient that decays from one end alone gets below the
# normal numbers, each of at most 2^12 steps rounds by up to 2^-150, gates below 1 carry that on,
# and states below 2^8 multiply it. (The values these tests are about are above 2^-94.)
UNDERFLOW = 2.0 ** -150 * 2.0 ** 12 * 2.0 ** 8


def _both_ways(monkeypatch, host, dev, dtype, what):
    """Parity with the oracle, and the same bits where every chunk computes for itself."""
    import torch
    ref = _oracle(host, dtype, False)
    got = _run(dev, False)
    _check(got, {k: (value, bound + UNDERFLOW) for k, (value, bound) in ref.items()}, what)
    monkeypatch.setenv("GS_RECURRENCE_PATIENCE", "0")
    alone = _run(dev, False)
    for k in ("h", "h_last", "ckpt", "grad_gate", "grad_x", "grad_h0"):
        assert torch.equal(got[k], alone[k]), (what, k)


@pytest.mark.parametrize("dtype,D", [("f32", 70), ("bf16", 70), ("bf16", 33)])
def test_gates_that_decay_and_grow_over_a_thousand_steps(monkeypatch, dtype, D):
    """Gates of 0.94 for 1024 steps, above 1 for 1024, 0.94 again: the states (and, from the other
    end, the gradients) stay between 1e-28 and 1e18, the product of the growing gates alone passes
    float32. Other channels have ordinary gates and inputs."""
    say(f"[recurrence decay and growth {dtype} D={D}]")
    T = 3000
    rng = np.random.default_rng(D)
    gate = np.full((T, D), 0.94)
    gate[1024:2048] = rng.uniform(1.092, 1.1, D)
    gate[:, D // 2:] = 1.0 / (1.0 + np.exp(-rng.normal(3.0, 1.5, (T, D - D // 2))))
    x = np.zeros((T, D))
    x[:, D // 2:] = rng.normal(0, 1, (T, D - D // 2))
    assert (np.prod(gate[1024:2048, :D // 2], 0) > 3.4e38).all()
    host, dev = _of_gates(dtype, gate, 1.0, 1.0, x)
    _both_ways(monkeypatch, host, dev, dtype, "growth")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_zero_gate_inside_a_growing_group(monkeypatch, dtype):
    """1.5^300 passes float32 (the state, 3e-28 in front, does not); a gate of 0 behind it ends
    what is left of the state, and what comes in later is there. Reversed in time for the gradients."""
    say(f"[recurrence zero gate {dtype}]")
    T, D = 2500, 65
    gate = np.full((T, D), 0.94)
    gate[1024:1324] = 1.5
    gate[1324] = 0.0
    x = np.zeros((T, D))
    x[1400:] = np.random.default_rng(1).normal(0, 1, (T - 1400, D))
    host, dev = _of_gates(dtype, gate, 1.0, 1.0, x)
    _both_ways(monkeypatch, host, dev, dtype, "forward")
    # from the end of 20 chunks the second group is steps 512 to 1535: growing from its end, then the zero
    T = 2560
    gate = np.full((T, D), 0.94)
    gate[T - 1324:T - 1024] = 1.5
    gate[T - 1325] = 0.0
    monkeypatch.delenv("GS_RECURRENCE_PATIENCE")
    host, dev = _of_gates(dtype, gate, 0.0, 1.0)
    _both_ways(monkeypatch, host, dev, dtype, "backward")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_large_state_outlives_a_product_that_underflows(monkeypatch, dtype):
    """0.89^1024 = 2e-52 is 0 in float32; a state of 1e37 in front of those steps is 2e-15 behind
    them. The same for the gradients' chain."""
    say(f"[recurrence large state {dtype}]")
    T, D = 3000, 65
    gate = np.ones((T, D))
    gate[1024:2048] = 0.89
    host, dev = _of_gates(dtype, gate, 1e37, 0.0)
    _both_ways(monkeypatch, host, dev, dtype, "forward")
    monkeypatch.delenv("GS_RECURRENCE_PATIENCE")
    host, dev = _of_gates(dtype, gate, 0.0, 1e37)
    _both_ways(monkeypatch, host, dev, dtype, "backward")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_states_of_ordinary_gates(monkeypatch, dtype, sigmoid):
    """States of 1e9 over gates whose product over 1024 steps is 0 in float32: what comes in later
    is as large, so nothing is lost with the product."""
    import torch
    say(f"[recurrence large states {dtype} sigmoid={sigmoid}]")
    host, dev = _inputs(12, 2, 3100, 66, dtype, sigmoid, ragged=True, restarts=True)
    for k in ("x", "grad_h", "h0", "grad_last"):
        dev[k] = dev[k] * 2.0 ** 30
        host[k] = to_np(dev[k].double())
    ref = _oracle(host, dtype, sigmoid)
    got = _run(dev, sigmoid)
    _check(got, ref, "large")
    monkeypatch.setenv("GS_RECURRENCE_PATIENCE", "0")
    alone = _run(dev, sigmoid)
    for k in ("h", "h_last", "grad_gate", "grad_x", "grad_h0"):
        assert torch.equal(got[k], alone[k]), k
