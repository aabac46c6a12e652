"""The float64 oracles of the delta rule and of the block norms against differences of their own outputs."""
import numpy as np
import pytest

from oracle import blocks


def _difference(call, args, name, direction, upstream, eps=1e-6):
    up, down = (dict(args, **{name: args[name] + s * eps * direction}) for s in (1, -1))
    a, b = call(**up), call(**down)
    return sum((upstream[k] * (a[k] - b[k])).sum() for k in upstream) / (2 * eps)


@pytest.mark.parametrize("ragged,restarts,group", [(False, False, 1), (True, True, 2)])
def test_delta_rule_gradients(ragged, restarts, group):
    rng = np.random.default_rng(3)
    B, T, Hk, dk, dv = 2, 9, 2, 5, 4
    H = Hk * group
    f = lambda *s: rng.standard_normal(s)  # noqa: E731
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    args = dict(q=unit(f(B, T, Hk, dk)), k=unit(f(B, T, Hk, dk)), v=f(B, T, H, dv), log_decay=-np.exp(f(B, T, H) - 1),
                beta=1 / (1 + np.exp(-f(B, T, H))), h0=f(B, H, dk, dv))
    fixed = dict(lengths=np.array([T, 6]) if ragged else None,
                 restart=(rng.random((B, T)) < 0.3).astype(np.uint8) if restarts else None)
    up = dict(o=f(B, T, H, dv), h_last=f(B, H, dk, dv))
    if ragged:
        up["o"][1, 6:] = 0
    got = blocks.delta_rule(**args, **fixed, grad_o=up["o"], grad_last=up["h_last"])
    for name in args:
        d = f(*args[name].shape)
        want = _difference(lambda **a: blocks.delta_rule(**a, **fixed), args, name, d, up)
        assert abs((got["grad_" + name] * d).sum() - want) < 1e-6 * (1 + abs(want)), name


@pytest.mark.parametrize("post,gating,pre", [("rms", "silu", "rms"), ("layer", "sigmoid", "layer"), ("none", "none", "rms"),
                                             ("rms", "silu", "none")])
def test_block_norm_gradients(post, gating, pre):
    rng = np.random.default_rng(4)
    f = lambda *s: rng.standard_normal(s)  # noqa: E731
    R, D = 3, 7
    args = dict(y=f(R, D), residual=f(R, D), gate=f(R, D), scale=f(D))
    if post != "none":
        args.update(post_weight=f(D), post_bias=f(D))
    if pre != "none":
        args.update(pre_weight=f(D), pre_bias=f(D))
    if gating == "none":
        del args["gate"]
    fixed = dict(post=post, gating=gating, pre=pre, eps=1e-3)
    up = dict(out=f(R, D))
    if pre != "none":
        up["norm"] = f(R, D)
    got = blocks.block_norm(**args, **fixed, grad_out=up["out"], grad_norm=up.get("norm"))
    for name in args:
        d = f(*args[name].shape)
        want = _difference(lambda **a: blocks.block_norm(**a, **fixed), args, name, d, up)
        assert abs((got["grad_" + name] * d).sum() - want) < 1e-6 * (1 + abs(want)), name


def test_off_counts_roundings():
    x = np.linspace(-3, 3, 101)
    assert blocks.off(x, x) == 0
    assert blocks.off(x * (1 + 2.0 ** -8), x, "bf16") <= 1
    assert blocks.off(x * (1 + 2.0 ** -8), x, "f32") > 1
    assert blocks.off(x * (1 + 2.0 ** -6), x, "bf16") > 1
