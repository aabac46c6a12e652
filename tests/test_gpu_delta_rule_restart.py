"""What is not finite in front of a restart (behind it, for gradients) ends there, however many steps a call has."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import blocks
from test_gpu_delta_rule import host, make, run

pytestmark = pytest.mark.gpu

# steps and restarts: at the first step, inside the first chunk, at a chunk's end, in a later chunk, in later segments
CASES = [(8, [0]), (9, [0]), (9, [5]), (100, [0]), (100, [37, 80]), (200, [63]), (200, [150]), (2100, [0]), (2100, [700]),
         (2100, [1300, 1301, 2050])]


def same(got, want, dtype, name):
    """Not finite where the oracle is not, and right elsewhere."""
    got = got.double().cpu().numpy()
    here = np.isfinite(want)
    assert (np.isfinite(got) == here).all(), (name, int((np.isfinite(got) != here).sum()))
    assert blocks.off(got[here], want[here], dtype) <= 1, name


def all_same(out, want, dtype):
    for n, w in want.items():
        same(out[n], w, dtype if n in ("o", "grad_q", "grad_k", "grad_v") else "f32", n)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["head", "channel", "element"])
@pytest.mark.parametrize("T,at", CASES)
def test_states_end_at_a_restart(T, at, kind, dtype):
    import torch
    d, up = make(2, T, 1, 2, 64, 48, dtype, T + len(at), restarts=True)
    d["restart"].zero_()
    d["restart"][:, at] = 1
    nan, inf = float("nan"), float("inf")
    part = (0, 0) if kind == "head" else (0, 0, slice(None), 3) if kind == "channel" else (0, 0, 2, 3)
    d["h0"][part] = inf if kind == "element" else nan
    up["grad_last"][(0, 1) + part[2:]] = -inf if kind == "element" else nan
    with np.errstate(invalid="ignore"):
        all_same(run(d, up), blocks.delta_rule(**host(d), **host(up)), dtype)
    clean, cup = dict(d, h0=d["h0"].clone()), dict(up, grad_last=up["grad_last"].clone())
    clean["h0"][part] = 0.0
    cup["grad_last"][(0, 1) + part[2:]] = 0.0
    if at[0] == 0:  # h0 is of no consequence at all
        got, want = run(d, cup), run(clean, cup)
        for n in want:
            assert n == "ckpt" or torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_drop_by_the_decay(dtype):
    """A decay that is 0 in float32 is a restart; decays whose product only is too small for it are none."""
    d, up = make(1, 150, 1, 2, 64, 48, dtype, 3)
    d["h0"][:] = float("nan")
    d["log_decay"][:, :, 0] = -3.0
    d["log_decay"][:, 90, 1] = -float("inf")
    out = run(d, up)
    assert not out["o"][:, :, 0].isfinite().any() and not out["h_last"][:, 0].isfinite().any()
    assert not out["grad_beta"][:, :, 0].isfinite().any()
    with np.errstate(invalid="ignore"):
        want = blocks.delta_rule(**host(d), **host(up))
    for n in ("o", "grad_q", "grad_k", "grad_v", "grad_beta", "grad_log_decay"):
        same(out[n][:, :, 1:] if out[n].shape[2] == 2 else out[n], want[n][:, :, 1:] if want[n].shape[2] == 2 else want[n],
             dtype if n in ("o", "grad_q", "grad_k", "grad_v") else "f32", n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 768])
def test_inputs_end_at_a_restart_of_another_chunk(shift, dtype):
    """A document with a value, or an upstream gradient, that is not finite spoils none behind (in front of) the chunk
    of the restart that ends it; shift: in segments."""
    d, up = make(1, 200 + 3 * shift, 1, 2, 64, 48, dtype, 17 + shift, restarts=True)
    d["restart"].zero_()
    d["restart"][:, [shift + 70, shift + 100]] = 1
    d["v"][0, 10, 0, 5] = float("nan")
    up["grad_o"][0, shift + 150, 0, 7] = float("inf")
    out = run(d, up)
    clean, cup = dict(d, v=d["v"].clone()), dict(up, grad_o=up["grad_o"].clone())
    clean["v"][0, 10], cup["grad_o"][0, shift + 150] = 0.0, 0.0
    want = blocks.delta_rule(**host(clean), **host(cup))
    doc = slice(shift + 70, shift + 100)
    for n in ("o", "grad_q", "grad_k", "grad_v", "grad_beta", "grad_log_decay"):
        got, w = out[n].double().cpu().numpy(), want[n]
        kind = dtype if n in ("o", "grad_q", "grad_k", "grad_v") else "f32"
        assert blocks.off(got[:, doc], w[:, doc], kind) <= 1, n
    assert blocks.off(out["o"].double().cpu().numpy()[:, shift + 70:], want["o"][:, shift + 70:], dtype) <= 1
    assert blocks.off(out["h_last"].cpu().numpy(), want["h_last"]) <= 1


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [8, 100, 2100])
def test_padding_stays_zero(T, dtype):
    """Outputs and gradients of padding are 0 whatever the states hold."""
    d, up = make(3, T, 1, 2, 64, 48, dtype, 23 + T, ragged=True)
    d["lengths"][:] = d["lengths"].new_tensor([T, max(T - 5, 1), 3])
    d["h0"][:, 1], up["grad_last"][:, 0] = float("nan"), float("inf")
    out = run(d, up)
    for b in range(3):
        n = int(d["lengths"][b])
        assert not out["o"][b, :n, 1].isfinite().any() and out["o"][b, :n, 0].isfinite().all()
        for k in ("o", "grad_q", "grad_k", "grad_v", "grad_log_decay", "grad_beta"):
            assert (out[k][b, n:] == 0).all(), (k, b)
