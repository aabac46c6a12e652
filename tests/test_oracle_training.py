"""The oracle of the sequence and training operators: its gradients against
central differences of its forward, its steps against closed forms."""
import numpy as np
import pytest

from oracle import training as tr


def _inputs(seed, B, T, D, sigmoid, ragged, restarts):
    rng = np.random.default_rng(seed)
    gate = rng.normal(1.0, 1.0, (B, T, D))
    if not sigmoid:
        gate = 1.0 / (1.0 + np.exp(-gate))
    x, h0 = rng.normal(0, 1, (B, T, D)), rng.normal(0, 1, (B, D))
    lengths = rng.integers(0, T + 1, B) if ragged else None
    if ragged:
        lengths[0] = T
    restart = (rng.random((B, T)) < 0.3).astype(np.uint8) if restarts else None
    return gate, x, h0, lengths, restart


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("ragged,restarts", [(False, False), (True, False), (False, True), (True, True)])
def test_recurrence_gradients_match_differences(sigmoid, ragged, restarts):
    B, T, D = 4, 6, 3
    gate, x, h0, lengths, restart = _inputs(5, B, T, D, sigmoid, ragged, restarts)
    rng = np.random.default_rng(6)
    g, gl = rng.normal(0, 1, (B, T, D)), rng.normal(0, 1, (B, D))
    kw = dict(sigmoid=sigmoid, lengths=lengths, restart=restart)
    out = tr.recurrence(gate, x, h0, grad_h=g, grad_last=gl, **kw)

    def loss(gate, x, h0):
        o = tr.recurrence(gate, x, h0, **kw)
        return np.sum(o["h"][0] * g) + np.sum(o["h_last"][0] * gl)

    d = 1e-6
    for name, which in (("grad_gate", 0), ("grad_x", 1), ("grad_h0", 2)):
        args = [gate, x, h0]
        num = np.zeros_like(args[which])
        for i in np.ndindex(num.shape):
            lo, hi = [a.copy() for a in args], [a.copy() for a in args]
            lo[which][i] -= d
            hi[which][i] += d
            num[i] = (loss(*hi) - loss(*lo)) / (2 * d)
        # central differences: d^2 times third derivatives (of order 10) plus rounding, 1e-16 * 100 / d
        np.testing.assert_allclose(out[name][0], num, atol=3e-7, rtol=0)


def test_recurrence_closed_forms():
    # a constant gate: h_t = a^(t+1) h0 + x (1 - a^(t+1)) / (1 - a)
    T, a, x, h0 = 9, 0.75, 0.5, 2.0
    o = tr.recurrence(np.full((1, T, 1), a), np.full((1, T, 1), x), np.full((1, 1), h0))
    t = np.arange(1, T + 1)
    np.testing.assert_allclose(o["h"][0][0, :, 0], a ** t * h0 + x * (1 - a ** t) / (1 - a), rtol=1e-14)
    # the convex form keeps a constant input
    o = tr.recurrence(np.linspace(-20, 20, T).reshape(1, T, 1), np.full((1, T, 1), x), np.full((1, 1), x), sigmoid=True)
    np.testing.assert_allclose(o["h"][0], x, rtol=1e-14)
    # length 0 hands the state on; a restart forgets it
    o = tr.recurrence(np.full((2, 3, 1), 1.0), np.zeros((2, 3, 1)), np.array([[5.0], [7.0]]), lengths=np.array([0, 3]),
                      restart=np.array([[0, 0, 0], [0, 1, 0]], np.uint8))
    np.testing.assert_array_equal(o["h_last"][0][:, 0], [5.0, 0.0])
    np.testing.assert_array_equal(o["h"][0][1, :, 0], [7.0, 0.0, 0.0])


def test_norm_clip_and_adam():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    assert tr.grad_norm(g) == 5.0 and tr.grad_norm(g, "max") == 4.0 and tr.grad_norm([]) == 0.0
    assert tr.clip_factor(0.5, 1.0) == 1.0 and abs(tr.clip_factor(2.0, 1.0) - 0.5) < 1e-6
    assert np.isnan(tr.clip_factor(np.nan, 1.0)) and tr.clip_factor(np.inf, 1.0) == 0.0
    # the first step from zero moments moves by lr against the gradient's sign, whatever its size
    p, m, v = tr.adam(np.zeros(3), np.array([1e-3, -5.0, 20.0]), np.zeros(3), np.zeros(3), 0, 0.1, 0.0, 0.9, 0.999, 1e-12)
    np.testing.assert_allclose(p, [-0.1, 0.1, -0.1], rtol=1e-8)
    # no gradient: only the decay
    p, _, _ = tr.adam(np.full(2, 3.0), np.zeros(2), np.zeros(2), np.zeros(2), 9, 0.1, 0.5, 0.9, 0.999, 1e-8)
    np.testing.assert_allclose(p, 3.0 * 0.95, rtol=1e-15)
