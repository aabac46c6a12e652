"""GPU tests of the gated linear recurrence at gates outside the ordinary range: NaN, and
logits at which the logistic function saturates. Inputs, oracle and bounds as in
test_gpu_recurrence.py."""
import numpy as np
import pytest

from gpu_helpers import to_np
from test_gpu_recurrence import _check, _inputs, _oracle, _run, _torch_type, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,D", [(1, 96), (3, 33), (20, 96), (128, 33), (400, 96)])
def test_nan_gate_reaches_what_it_should(dtype, sigmoid, T, D):
    """A NaN gate at step s: every state from s on, the gate's gradient at every step (through the
    state behind s, through d in front of it), the input's gradient in front of s (at s too
    where the gate scales the input) and grad_h0 are NaN; nothing of another channel is."""
    import gaussian_splatting_tile_amd as gs
    say(f"[recurrence NaN gate {dtype} sigmoid={sigmoid} {T}x{D}]")
    _, dev = _inputs(T, 1, T, D, dtype, sigmoid)
    s, ch = T // 2, 7
    dev["gate"][0, s, ch] = float("nan")
    out = _run(dev, sigmoid)
    got = {k: to_np(v.double()) for k, v in out.items()}
    nan = {k: np.zeros(got[k].shape, bool) for k in ("h", "h_last", "grad_gate", "grad_x", "grad_h0")}
    nan["h"][0, s:, ch] = nan["h_last"][0, ch] = nan["grad_h0"][0, ch] = True
    nan["grad_gate"][0, :s, ch] = nan["grad_x"][0, :s, ch] = nan["grad_gate"][0, s + 1:, ch] = True
    if sigmoid:
        nan["grad_gate"][0, s, ch] = nan["grad_x"][0, s, ch] = True
    for k, want in nan.items():
        bad = np.isnan(got[k]) != want
        assert not bad.any(), (k, np.argwhere(bad)[:3].tolist())
        assert np.isfinite(got[k][~want]).all(), k
    # so a step that skips non-finite gradients sees it
    assert np.isnan(float(gs.grad_norm([out["grad_gate"], out["grad_x"], out["grad_h0"]])))

# Logits around and past the ends of float32's exponential (|z| = 87.3 to 104), and far past them.
EXTREMES = [np.inf, 1e4, 200.0, 104.0, 100.0, 89.0, 88.0, 87.4, 87.3, 86.6, 86.5, 80.0]
# What a flush of results below the smallest normal number, 2^-126, may be off by: that much times
# the sum over at most 2^10 steps of products of three states, inputs or gradients, each below 2^5.
FLUSH = 2.0 ** -126 * 2.0 ** 10 * 2.0 ** 15


def _saturate(seed, dtype, B, T, D):
    """Half the gates at an extreme of either sign. In the oracle's inputs they end at 200: its
    logistic function is 1e-87 away from 0 or 1 there, and its bound grows with the logit."""
    import torch
    host, dev = _inputs(seed, B, T, D, dtype, True)
    rng = np.random.default_rng(seed + 1)
    gate = np.where(rng.random((B, T, D)) < 0.5, rng.choice(EXTREMES + [-z for z in EXTREMES], (B, T, D)), host["gate"])
    dev["gate"] = torch.from_numpy(gate).to(_torch_type(dtype)).cuda()
    dev["x"][rng.random((B, T, D)) < 0.1] = 0.0
    host["gate"] = np.clip(to_np(dev["gate"].double()), -200.0, 200.0)
    host["x"] = to_np(dev["x"].double())
    return host, dev


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,T,D", [(3, 1, 96), (3, 1, 33), (2, 3, 64), (2, 20, 130), (2, 128, 33), (1, 700, 96)])
def test_saturated_gates_parity(dtype, B, T, D):
    say(f"[recurrence saturated gates {dtype} {B}x{T}x{D}]")
    host, dev = _saturate(T + D, dtype, B, T, D)
    ref = _oracle(host, dtype, True)
    out = _run(dev, True)
    _check(out, {k: (value, bound + FLUSH) for k, (value, bound) in ref.items()}, (dtype, T))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gate", [-np.inf, -1e4, -200.0])
@pytest.mark.parametrize("T", [1, 3, 20, 300])
def test_a_forced_forget_is_a_forget(dtype, gate, T):
    """sigmoid(gate) is 0 and 1 - sigmoid(gate) is 1 to float32: the state is the input, its
    gradient the upstream one, and nothing is left of the state in front."""
    import torch
    say(f"[recurrence forget {dtype} gate={gate} T={T}]")
    host, dev = _inputs(T, 2, T, 70, dtype, True)
    dev["gate"].fill_(gate)
    dev["x"][:, :, 1] = 0.0
    dev["h0"].fill_(1e30)
    out = _run(dev, True)
    assert torch.equal(out["h"], dev["x"]) and torch.equal(out["h_last"], dev["x"][:, -1].float())
    want = dev["grad_h"].float()
    want[:, -1] += dev["grad_last"]
    assert torch.equal(out["grad_x"], want.to(dev["x"].dtype))
    assert not out["grad_gate"].any() and not out["grad_h0"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gate", [np.inf, 1e4, 200.0])
@pytest.mark.parametrize("T", [1, 3, 20, 300])
def test_a_forced_keep_is_a_keep(dtype, gate, T):
    """sigmoid(gate) is 1 and 1 - sigmoid(gate) is 0: the state stays h0 whatever comes in."""
    import torch
    say(f"[recurrence keep {dtype} gate={gate} T={T}]")
    host, dev = _inputs(T, 2, T, 70, dtype, True)
    dev["gate"].fill_(gate)
    out = _run(dev, True)
    assert torch.equal(out["h"], dev["h0"].to(dev["x"].dtype)[:, None].expand(2, T, 70))
    assert torch.equal(out["h_last"], dev["h0"])
    assert not out["grad_gate"].any() and not out["grad_x"].any()
