"""GPU tests of the gated linear recurrence's state across chunks of steps: one buffer for the
state in front and behind, however the chunks get it. Inputs and oracle as in
test_gpu_recurrence.py."""
import pytest

from test_gpu_recurrence import _inputs, _run, say

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
