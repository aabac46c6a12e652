"""GPU tests of the gated linear recurrence at gates outside the ordinary range: NaN.
Inputs, oracle and bounds as in
test_gpu_recurrence.py."""
import numpy as np
import pytest

from gpu_helpers import to_np
from test_gpu_recurrence import _inputs, _run, say

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
