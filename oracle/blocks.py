"""Plain float64 implementations of the gated delta rule and of the norms
around a block, from their definitions. Test infrastructure only; shares no
code with the library.

Tolerances (TOL, close). u = 2^-24 is float32's unit roundoff. An output of
either operator is behind at most 8 dependent sums of products, each of n <= 192
terms (128 of a state's dimension and 64 of a chunk's steps), whose roundings
of at most u relative to the running sum have either sign: u sqrt(n / 3) =
4.8e-7 of the sum's size a stage, in quadrature over 8 stages 1.4e-6, and twice
that where a difference cancels: 2^-18 = 3.8e-6 of an output's root mean square,
in the root mean square over the output. Gates and keys are chosen so that no
stage amplifies (decays at most 1, unit keys, beta at most 1). A single element
may be off by 16 such deviations; the rounding to a 16-bit type adds half a
unit in its last place, at least half its smallest subnormal. A norm's sums are
longer (16384 terms), but each thread adds at most 16 of them one by one and
the rest as a tree, so the same bound holds for them.

LOST is what a bfloat16 output of the delta rule may lack beside that, as a
part of the root of the sum of its terms' squares ("terms" of delta_rule):
nothing, as the bound above holds before the rounding to any type.
"""
from __future__ import annotations

import numpy as np

TOL = 2.0 ** -18
LOST = 0.0
# unit roundoff and half of the smallest subnormal
TYPES = {"f32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}


def off(got, want, dtype="f32", sums=1.0, size=0.0, lost=0.0):
    """How many times further `got` is from `want` than it may be: at most 1 is right. `sums`: how many times longer
    than 192 terms an output's sums are, as a factor of the bound. `size`: the root mean square of terms whose
    difference the output is, each rounded by itself, where it is more than the output's. `lost`: what may be missing
    of a value in any case, as numbers too small for float32 are."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    if not want.size:
        return 0.0
    assert np.isfinite(got).all()
    u, tiny = TYPES[dtype]
    rms = max(np.sqrt(np.mean(want * want)), size)
    err = np.maximum(np.abs(got - want) - u * np.abs(want) - tiny - lost, 0.0)
    worst = err.max() / (16 * TOL * sums * rms + 1e-300)
    return max(worst, np.sqrt(np.mean(err * err)) / (TOL * sums * rms + 1e-300))


def delta_rule(q, k, v, log_decay, beta, h0=None, scale=None, lengths=None, restart=None, grad_o=None, grad_last=None,
               terms=False):
    """gs_delta_rule_fwd, and gs_delta_rule_bwd when grad_o is given, step by step. Returns a dict."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    r = H // Hk
    scale = dk ** -0.5 if scale is None else scale
    S = np.zeros((B, H, dk, dv)) if h0 is None else h0.astype(np.float64)
    n = np.full((B,), T) if lengths is None else np.clip(lengths, 0, T)
    live = np.arange(T)[None, :] < n[:, None]
    drop = np.zeros((B, T), bool) if restart is None else restart != 0
    wide = lambda x: np.repeat(np.where(live[:, :, None, None], x, 0.0).astype(np.float64), r, axis=2)  # noqa: E731
    q, k = scale * wide(q), wide(k)
    v = np.where(live[:, :, None, None], v, 0.0).astype(np.float64)
    alpha = np.where(live[:, :, None], np.exp(np.where(live[:, :, None], log_decay, 0.0).astype(np.float64)), 1.0)
    alpha = np.where((drop & live)[:, :, None], 0.0, alpha)
    beta = np.where(live[:, :, None], beta, 0.0).astype(np.float64)
    o = np.zeros((B, T, H, dv))
    before, errs, states = [], [], []
    for t in range(T):
        before.append(S)
        # a dropped state is dropped whatever it holds
        D = np.where(alpha[:, t, :, None, None] == 0.0, 0.0, alpha[:, t, :, None, None] * S)
        e = v[:, t] - np.einsum("bhkv,bhk->bhv", D, k[:, t])
        S = D + k[:, t, :, :, None] * (beta[:, t, :, None] * e)[:, :, None, :]
        errs.append(e)
        states.append(S)
        o[:, t] = np.einsum("bhkv,bhk->bhv", S, q[:, t])
    out = dict(o=o, h_last=S)
    if terms:
        size = np.zeros_like(o)
        for t in range(T):
            c = t - t % 64
            a = np.concatenate([np.cumprod(alpha[:, t:c:-1], 1)[:, ::-1], np.ones((B, 1, H))], 1)  # behind j, j = c .. t
            front = alpha[:, c] * a[:, 0]
            size[:, t] = np.einsum("bhkv,bhk->bhv", before[c] ** 2, q[:, t] ** 2) * front[..., None] ** 2
            p = a * np.einsum("bjhk,bhk->bjh", k[:, c:t + 1], q[:, t])
            u = beta[:, c:t + 1, :, None] * np.stack(errs[c:t + 1], 1)
            size[:, t] += np.einsum("bjh,bjhv->bhv", p ** 2, u ** 2)
        out["terms"] = np.sqrt(size)
    if grad_o is None:
        return out
    go = np.where(live[:, :, None, None], grad_o, 0.0).astype(np.float64)
    dS = np.zeros_like(S) if grad_last is None else grad_last.astype(np.float64)
    dq, dk_, dv_, dg, db = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(beta), np.zeros_like(beta)
    for t in range(T - 1, -1, -1):
        a, b = alpha[:, t, :, None, None], beta[:, t, :, None]
        dq[:, t] = scale * np.einsum("bhkv,bhv->bhk", states[t], go[:, t])
        dS = dS + q[:, t, :, :, None] * go[:, t, :, None, :]
        du = np.einsum("bhkv,bhk->bhv", dS, k[:, t])
        D = np.where(a == 0.0, 0.0, a * before[t])
        dk_[:, t] = np.einsum("bhkv,bhv->bhk", dS, b * errs[t]) - np.einsum("bhkv,bhv->bhk", D, b * du)
        dv_[:, t] = b * du
        db[:, t] = (du * errs[t]).sum(-1)
        dS = dS - k[:, t, :, :, None] * (b * du)[:, :, None, :]
        dg[:, t] = np.where(a == 0.0, 0.0, dS * D).sum((-1, -2))
        dS = np.where(a == 0.0, 0.0, a * dS)
    m, m1 = live[:, :, None], live[:, :, None, None]
    shared = lambda x: np.where(m1, x, 0.0).reshape(B, T, Hk, r, dk).sum(3)  # noqa: E731
    out.update(grad_q=shared(dq), grad_k=shared(dk_), grad_v=np.where(m1, dv_, 0.0), grad_log_decay=np.where(m, dg, 0.0),
               grad_beta=np.where(m, db, 0.0), grad_h0=dS)
    return out


def _normed(x, kind, eps):
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r, r


def _normed_back(g, xhat, r, kind):
    d = g - xhat * (g * xhat).mean(-1, keepdims=True)
    if kind == "layer":
        d = d - g.mean(-1, keepdims=True)
    return r * d


def block_norm(y, residual=None, gate=None, gating="none", scale=None, post="none", post_weight=None, post_bias=None,
               pre="none", pre_weight=None, pre_bias=None, eps=1e-6, grad_out=None, grad_norm=None):
    """gs_block_norm_fwd, and gs_block_norm_bwd when a gradient is given. Returns a dict; its "sizes" are those of the
    cancelling terms of gradients, for off()."""
    f = lambda x, d: d if x is None else np.asarray(x, np.float64)  # noqa: E731
    y, w, b, s, w2, b2 = f(y, 0), f(post_weight, 1.0), f(post_bias, 0.0), f(scale, 1.0), f(pre_weight, 1.0), f(pre_bias, 0.0)
    yhat, r = _normed(y, post, eps) if post != "none" else (y, 1.0)
    t = yhat * w + b
    act = slope = np.ones_like(y)
    if gating != "none":
        z = f(gate, 0)
        sg = 1.0 / (1.0 + np.exp(-z))
        act, slope = (sg, sg * (1 - sg)) if gating == "sigmoid" else (z * sg, sg * (1 + z * (1 - sg)))
    c = act * t
    x = s * c + f(residual, 0.0)
    out = dict(out=x)
    if pre != "none":
        xhat, r2 = _normed(x, pre, eps)
        out["norm"] = xhat * w2 + b2
    if grad_out is None and grad_norm is None:
        return out
    cols = lambda v: v.reshape(-1, v.shape[-1]).sum(0)  # noqa: E731
    d = np.zeros_like(y) if grad_out is None else np.asarray(grad_out, np.float64)
    # a norm's gradient is a difference: the size of its terms, r g, as one number for the call
    sizes = {}
    if pre != "none":
        g = np.asarray(grad_norm, np.float64)
        out.update(grad_pre_weight=cols(g * xhat), grad_pre_bias=cols(g))
        sizes["grad_residual"] = np.sqrt(np.mean((r2 * g * w2) ** 2))
        d = d + _normed_back(g * w2, xhat, r2, pre)
    out.update(grad_residual=d, grad_scale=cols(d * c))
    d = d * s
    out["grad_gate"] = d * t * slope
    d = d * act
    sizes["grad_y"] = np.sqrt(np.mean((r * d * w) ** 2))
    if post != "none":
        out.update(grad_post_weight=cols(d * yhat), grad_post_bias=cols(d))
        d = _normed_back(d * w, yhat, r, post)
    out["grad_y"] = d
    out["sizes"] = sizes
    return out
