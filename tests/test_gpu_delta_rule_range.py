"""The gated delta rule on the GPU where values are far from 1: it is linear in the values and the first state, and in
the upstream gradients, so a power of two on them is one on the outputs, to the last bit."""
from __future__ import annotations

import pytest

from oracle import blocks
from test_gpu_delta_rule import host, make, run

pytestmark = pytest.mark.gpu

# chunks of one workgroup, one boundary between chunks, several with lengths that differ, and segments
CASES = [(2, 65, 1, 2, 64, 48, ""), (3, 200, 2, 4, 128, 128, "lr"), (1, 2100, 1, 2, 64, 80, ""), (2, 2100, 1, 1, 128, 64, "r")]


def moderate(d):
    """Decays of which no product over a chunk is near float32's smallest, so that powers of two stay exact; those of
    the last head close to 1."""
    d["log_decay"].clamp_(min=-0.3)
    d["log_decay"][:, :, -1] *= 1e-3


def scaled(d, up, by, up_by):
    """The inputs with values, states and upstream gradients times powers of two (numbers, or one a value channel)."""
    d, up = dict(d), dict(up)
    for x, names, f in ((d, ("v", "h0"), by), (up, ("grad_o", "grad_last"), up_by)):
        for n in names:
            if n in x:
                x[n] = (x[n] * f).to(x[n].dtype)
    return d, up


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("B,T,Hk,H,dk,dv,flags", CASES)
def test_powers_of_two(B, T, Hk, H, dk, dv, flags, state, dtype):
    import torch
    d, up = make(B, T, Hk, H, dk, dv, dtype, 3 * T + dk, "l" in flags, "r" in flags, state=state)
    moderate(d)
    if not state:
        del up["grad_last"]
    want = run(d, up)
    for a, b in ((20, 0), (0, 20), (10, 30), (-12, 24)):
        got = run(*scaled(d, up, 2.0 ** -a, 2.0 ** -b))
        for names, by in ((("o", "h_last"), a), (("grad_v", "grad_h0"), b),
                          (("grad_q", "grad_k", "grad_log_decay", "grad_beta"), a + b)):
            for n in names:
                assert torch.equal(got[n].double() * 2.0 ** by, want[n].double()), (n, a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("B,T,Hk,H,dk,dv,flags", CASES)
def test_channels_of_other_sizes(B, T, Hk, H, dk, dv, flags, state, dtype):
    """A value channel's outputs follow from that channel alone, so one that is small beside its neighbours, or has a
    first state of zeros beside others that have none, loses nothing."""
    import torch
    d, up = make(B, T, Hk, H, dk, dv, dtype, 5 * T + dk, "l" in flags, "r" in flags, state=state)
    moderate(d)
    if state:
        d["h0"][..., 2::7] = 0.0
        up["grad_last"][..., 4::7] = 0.0
    else:
        del up["grad_last"]
    f = torch.exp2(torch.arange(dv, device="cuda") % 7 * -5.0)
    want, got = run(d, up), run(*scaled(d, up, f, f))
    for n in ("o", "h_last", "grad_v", "grad_h0"):
        assert torch.equal(got[n].double() / f.double(), want[n].double()), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [130, 2100])
def test_small_values_against_oracle(T, dtype):
    """A step of training as it begins: no first state, no gradient of the last, small values and gradients of a mean,
    heads that forget slowly. Each head by itself."""
    import torch
    d, up = make(1, T, 1, 3, 64, 64, dtype, T, state=False)
    del up["grad_last"]
    d["log_decay"] *= torch.tensor([1.0, 1e-2, 1e-4], device="cuda")
    d, up = scaled(d, up, 2.0 ** -14, 2.0 ** -22)
    out, want = run(d, up), blocks.delta_rule(**host(d), **host(up), terms=True)
    for n in ("o", "h_last", "grad_v", "grad_h0", "grad_log_decay", "grad_beta"):
        kind = dtype if n in ("o", "grad_v") else "f32"
        for h in range(3):
            at = (slice(None), h) if n in ("h_last", "grad_h0") else (slice(None), slice(None), h)
            lost = blocks.LOST * want["terms"][at] if n == "o" and dtype == "bf16" else 0.0
            assert blocks.off(out[n].double().cpu().numpy()[at], want[n][at], kind, lost=lost) <= 1, (n, h)


@pytest.mark.parametrize("T", [9, 200, 2100])
def test_sixteen_bits_round_once(T):
    """A 16-bit output is a float32 one rounded at the end: no product is formed from fewer bits for it."""
    for dtype in ("bf16", "f16"):
        d, _ = make(1, T, 2, 4, 128, 128, dtype, 7 + T, train=False)
        o = run(d, {})["o"].double().cpu().numpy()
        assert blocks.off(o, blocks.delta_rule(**host(d))["o"], dtype) <= 1, dtype


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dv", [16, 40, 50, 128])
@pytest.mark.parametrize("T", [60, 130])
def test_key_dimensions_of_other_sizes(T, dv, dtype):
    """Gradients of key dimensions whose rows of the state and of its gradient are small beside the rows next to them:
    what those hold is no part of them. Queries and keys are 0 there, so that nothing else is in these gradients."""
    d, up = make(1, T, 1, 2, 64, dv, dtype, 3 * T + dv)
    moderate(d)
    for n in ("q", "k"):
        d[n][..., 1::2] = 0.0
    d["h0"][:, :, 1::2] *= 2.0 ** -20
    up["grad_last"][:, :, 1::2] *= 2.0 ** -20
    d, up = (d, up) if dtype != "f16" else scaled(d, up, 2.0 ** 4, 2.0 ** 4)  # float16's gradients stay clear of subnormals
    out, want = run(d, up), blocks.delta_rule(**host(d), **host(up))
    for n in ("grad_q", "grad_k"):
        for at in (slice(0, None, 2), slice(1, None, 2)):
            assert blocks.off(out[n].double().cpu().numpy()[..., at], want[n][..., at], dtype) <= 1, (n, at)


@pytest.mark.parametrize("T,train", [(1, True), (8, False)])
def test_wide_steps_of_short_calls(T, train):
    """Steps of more than 2^22 elements, as of the tokens of many sequences, in calls that address no chunk by them."""
    import torch
    d, up = make(2, T, 1, 2, 32, 48, "bf16", 41, train=train)
    wide = (1 << 22) + 64
    buffer = torch.empty(T * wide, dtype=torch.bfloat16, device="cuda")
    e, at = dict(d), 0
    for n in ("q", "k", "v"):
        B, _, H, dim = d[n].shape
        e[n] = buffer.as_strided(d[n].shape, (H * dim, wide, dim, 1), at)
        e[n].copy_(d[n])
        at += B * H * dim
    got, want = run(e, up), run(d, up)
    for n in want:
        assert got[n] is None or torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,decay", [(2, -18.0), (2, -1.0), (64, -12.0), (130, -9.0)])
def test_gradients_of_strong_decays(T, decay, dtype):
    """The gradient of a decay is a sum of what it reaches over: where it lets little through it is small beside the
    sums of the steps themselves, which are no part of it. (A restart at the first step leaves no state to the others.)"""
    d, up = make(4, T, 16, 16, 64, 64, dtype, T, restarts=True, state=False)
    del up["grad_last"]
    d["restart"].zero_()
    d["restart"][:, 0] = 1
    d["log_decay"].fill_(decay)
    got, want = run(d, up)["grad_log_decay"].double().cpu().numpy(), blocks.delta_rule(**host(d), **host(up))["grad_log_decay"]
    for t in range(1, T):
        assert blocks.off(got[:, t], want[:, t]) <= 1, t
