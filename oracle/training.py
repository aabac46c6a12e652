"""Plain float64 implementations of the sequence and training operators
(gated linear recurrence, global gradient norm and clipping, Adam), step by
step from their definitions, with bounds of what float32 arithmetic may be
off by. Test infrastructure only; shares no code with the library.

Bounds. eps = 2^-24 is float32's unit roundoff. The recurrence is evaluated
in some grouping of h_t = a_t h_{t-1} + u_t (products of gates over a chunk,
then one product with the state in front). Let M_t = |a_t| M_{t-1} + |u_t|
be the same recurrence on magnitudes. Whatever the grouping, a term
u_s a_{s+1} ... a_t passes at most one rounding per gate it is multiplied
with and one per addition on its way, so an error of c eps M_t enters at
step t and later gates carry it on: E_t = |a_t| E_{t-1} + c_t eps M_t with
c_t = 4 (two roundings of the step itself, two of a regrouped product and
sum), plus the relative error of a_t and u_t where they are computed: the
logistic function by a hardware exponential of z log2(e) is off by
(2 |z| + 8) eps. One rounding to the output's type comes on top: half a unit
in its last place, at least half its smallest subnormal.
"""
from __future__ import annotations

import numpy as np

EPS = 2.0 ** -24
# unit roundoff and half of the smallest subnormal
TYPES = {"f32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}


def stored(value, bound, dtype):
    """The bound after one rounding of `value` +- bound to dtype."""
    u, tiny = TYPES[dtype]
    return bound + u * (np.abs(value) + bound) + tiny


def _terms(gate, x, sigmoid):
    """a, u, 1 - a and the relative error (in eps) of the computed ones."""
    if not sigmoid:
        return gate, x, np.ones_like(gate), np.zeros_like(gate)
    e = np.exp(-np.abs(gate))
    big, small = 1.0 / (1.0 + e), e / (1.0 + e)
    a, rest = np.where(gate >= 0, big, small), np.where(gate >= 0, small, big)
    return a, rest * x, rest, 2.0 * np.abs(gate) + 8.0


def recurrence(gate, x, h0=None, sigmoid=False, lengths=None, restart=None, grad_h=None, grad_last=None, dtype="f32"):
    """Values and error bounds of gs_recurrence_fwd, and of gs_recurrence_bwd when grad_h is
    given. Arrays [B, T, D]; returns {name: (value, bound)}."""
    B, T, D = gate.shape
    gate, x = gate.astype(np.float64), x.astype(np.float64)
    h = np.zeros((B, D)) if h0 is None else h0.astype(np.float64)
    n = np.full((B,), T) if lengths is None else np.clip(lengths, 0, T)
    live = np.arange(T)[None, :] < n[:, None]
    keep = np.ones((B, T), bool) if restart is None else restart == 0
    # padding is never looked at, whatever it holds
    gate, x = np.where(live[:, :, None], gate, 0.0), np.where(live[:, :, None], x, 0.0)
    a, u, rest, ra = _terms(gate, x, sigmoid)
    M, E = np.abs(h), np.zeros((B, D))
    hs, Es, prev, Ep, Mp = (np.zeros((B, T, D)) for _ in range(5))
    for t in range(T):
        k = keep[:, t, None]
        p, q, mp = np.where(k, h, 0.0), np.where(k, E, 0.0), np.where(k, M, 0.0)
        prev[:, t], Ep[:, t], Mp[:, t] = p, q, mp
        at, l = a[:, t], live[:, t, None]
        m = np.abs(at) * mp + np.abs(u[:, t])
        M = np.where(l, m, M)
        E = np.where(l, np.abs(at) * q + (4.0 + ra[:, t]) * EPS * m, E)
        h = np.where(l, at * p + u[:, t], h)
        hs[:, t], Es[:, t] = np.where(l, h, 0.0), np.where(l, E, 0.0)
    out = dict(h=(hs, stored(hs, Es, dtype)), h_last=(h, E + EPS * np.abs(h)))
    if grad_h is None:
        return out
    g = np.where(live[:, :, None], grad_h.astype(np.float64), 0.0)
    c = np.zeros((B, D)) if grad_last is None else grad_last.astype(np.float64)
    Mc, Ec = np.abs(c), np.zeros((B, D))
    dg, dx, Eg, Ex = (np.zeros((B, T, D)) for _ in range(4))
    for t in range(T - 1, -1, -1):
        l, k = live[:, t, None], keep[:, t, None]
        d, Md = g[:, t] + c, np.abs(g[:, t]) + Mc
        Ed = Ec + 4.0 * EPS * Md
        at, r, rel = a[:, t], rest[:, t], ra[:, t]
        if sigmoid:
            w, Mw = prev[:, t] - x[:, t], Mp[:, t] + np.abs(x[:, t])
            s = at * r
            dg[:, t] = d * w * s
            Eg[:, t] = s * (Ed * np.abs(w) + np.abs(d) * (Ep[:, t] + EPS * Mw) + (2 * rel + 4) * EPS * np.abs(d * w))
            dx[:, t] = d * r
            Ex[:, t] = r * (Ed + (rel + 1) * EPS * np.abs(d))
        else:
            dg[:, t] = d * prev[:, t]
            Eg[:, t] = Ed * np.abs(prev[:, t]) + np.abs(d) * Ep[:, t] + EPS * np.abs(dg[:, t])
            dx[:, t], Ex[:, t] = d, Ed
        cn = np.where(k, at * d, 0.0)
        Mn = np.where(k, np.abs(at) * Md, 0.0)
        En = np.where(k, np.abs(at) * Ed, 0.0) + (4.0 + rel) * EPS * Mn
        c, Mc, Ec = np.where(l, cn, c), np.where(l, Mn, Mc), np.where(l, En, Ec)
    dg, dx = np.where(live[:, :, None], dg, 0.0), np.where(live[:, :, None], dx, 0.0)
    Eg, Ex = np.where(live[:, :, None], Eg, 0.0), np.where(live[:, :, None], Ex, 0.0)
    out.update(grad_gate=(dg, stored(dg, Eg, dtype)), grad_x=(dx, stored(dx, Ex, dtype)),
               grad_h0=(c, Ec + EPS * np.abs(c)))
    return out


def grad_norm(grads, kind="l2"):
    """The global norm of a list of arrays, in float64."""
    flat = np.concatenate([np.asarray(g, np.float64).reshape(-1) for g in grads]) if grads else np.zeros(0)
    if kind == "max":
        return np.abs(flat).max() if flat.size else 0.0
    return np.sqrt(np.sum(flat * flat))


def clip_factor(norm, max_norm):
    c = max_norm / (norm + 1e-6)
    return 1.0 if c > 1.0 else c


def adam(param, grad, m, v, step, lr, weight_decay, beta1, beta2, eps, factor=1.0):
    """One update of one tensor; `step` counts the updates taken before. Returns p, m, v."""
    g = factor * np.asarray(grad, np.float64)
    m = beta1 * np.asarray(m, np.float64) + (1.0 - beta1) * g
    v = beta2 * np.asarray(v, np.float64) + (1.0 - beta2) * g * g
    t = step + 1
    p = np.asarray(param, np.float64)
    p = p * (1.0 - lr * weight_decay) - lr * (m / (1.0 - beta1 ** t)) / (np.sqrt(v / (1.0 - beta2 ** t)) + eps)
    return p, m, v
