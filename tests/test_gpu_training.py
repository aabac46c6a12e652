"""GPU parity of the global gradient norm, clipping and the Adam update
(gs_grad_norm, gs_clip_grads, gs_adam_step) against float64, within the
roundings that float32 arithmetic makes on each element (eps = 2^-24):

  * norm: squares and sums in float64 (N 2^-53 relative), one rounding to
    float32;
  * clipped gradients: the factor's rounding, the product's, and one to the
    type: (2 eps + u) |out|;
  * Adam: see _adam_bounds.
"""
import sys

import numpy as np
import pytest

from gpu_helpers import to_np
from oracle import training as tr

pytestmark = pytest.mark.gpu
EPS = tr.EPS


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def _torch_type(dtype):
    import torch
    return dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[dtype]


def _grads(seed, sizes, dtypes, scale=1.0):
    """Slices of one arena per type: their starts are as odd as the sizes."""
    import torch
    rng = np.random.default_rng(seed)
    out = []
    for d in sorted(set(dtypes)):
        mine = [i for i in range(len(sizes)) if dtypes[i] == d]
        arena = torch.from_numpy(rng.normal(0, scale, sum(sizes[i] for i in mine))).to(_torch_type(d)).cuda()
        at = 0
        for i in mine:
            out.append((i, arena[at:at + sizes[i]]))
            at += sizes[i]
    return [t for _, t in sorted(out, key=lambda p: p[0])]


LISTS = {
    "one": [1],
    "few": [3, 1, 0, 4097, 64],
    "mlp": [2048, 64, 192, 3],
    "edges": [4095, 4096, 4097, 8192, 1023, 5, 16385],
    "many": [1 + (37 * k) % 311 for k in range(300)],
    "large": [3_000_001, 7, 500_000],
    "just over": [9_437_184 + 1],
}
MIXES = {"f32": ["f32"], "bf16": ["bf16"], "f16": ["f16"], "mixed": ["f32", "bf16", "f16", "bf16"]}


def _types(mix, n):
    return [MIXES[mix][i % len(MIXES[mix])] for i in range(n)]


def _close(got, want, bound, what):
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3])


@pytest.mark.parametrize("mix", sorted(MIXES))
@pytest.mark.parametrize("which", sorted(LISTS))
def test_norm_and_clip_parity(which, mix):
    import torch
    import gaussian_splatting_tile_amd as gs
    say(f"[norm {which} {mix}]")
    sizes = LISTS[which]
    types = _types(mix, len(sizes))
    grads = _grads(len(sizes), sizes, types)
    host = [to_np(g.double()) for g in grads]
    N = sum(sizes)
    outs = [torch.full_like(g, 7.0) for g in grads]
    lst = gs.GradList(grads, out=outs)
    for kind, name in ((gs.NORM_L2, "l2"), (gs.NORM_MAX, "max")):
        want = tr.grad_norm(host, name)
        tol = want * (EPS + N * 2.0 ** -53) if name == "l2" else 0.0
        assert abs(float(lst.norm(kind)) - want) <= tol, (name, float(lst.norm(kind)), want)
        for max_norm in (0.25 * want, 4.0 * want):
            max_norm = float(np.float32(max_norm))
            n = lst.clip(max_norm, kind)
            torch.cuda.synchronize()
            assert abs(float(n) - want) <= tol
            c = tr.clip_factor(want, max_norm)
            for g, o, h, d in zip(grads, outs, host, types):
                if c == 1.0:
                    assert torch.equal(g, o)
                else:
                    _close(to_np(o.double()), h * c, tr.stored(h * c, 3 * EPS * np.abs(h * c), d), (name, max_norm))
    # in place
    gs.GradList(grads).clip(0.5 * float(tr.grad_norm(host)) + 1e-3)
    torch.cuda.synchronize()
    c = tr.clip_factor(tr.grad_norm(host), np.float32(0.5 * float(tr.grad_norm(host)) + 1e-3))
    for g, h, d in zip(grads, host, types):
        _close(to_np(g.double()), h * c, tr.stored(h * c, 3 * EPS * np.abs(h * c), d), "in place")


@pytest.mark.parametrize("name", ["mlp", "large"])
def test_clip_in_place_below_the_norm_keeps_the_bits(name):
    """A factor of 1: gradients in place stay as they are, others are copied; above the
    norm's bound the same list is scaled everywhere."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[clip in place]", name)
    types = _types("mixed", len(LISTS[name]))
    grads = _grads(7, LISTS[name], types)
    grads[0][:3] = torch.tensor([-0.0, 1e-40, 0.0])  # (1e-40 is subnormal)
    before = [g.clone() for g in grads]
    outs = [g if i % 2 == 0 else torch.full_like(g, 7.0) for i, g in enumerate(grads)]
    norm = tr.grad_norm([to_np(g.double()) for g in grads])
    lst = gs.GradList(grads, out=outs)
    lst.clip(float(4.0 * norm))
    torch.cuda.synchronize()
    for g, o, b in zip(grads, outs, before):
        bits = torch.int32 if g.dtype == torch.float32 else torch.int16
        assert torch.equal(g.view(bits), b.view(bits)) and torch.equal(o.view(bits), b.view(bits))
    lst.clip(float(0.5 * norm))
    torch.cuda.synchronize()
    c = tr.clip_factor(norm, np.float32(0.5 * norm))
    for o, b, d in zip(outs, before, types):
        h = to_np(b.double())
        _close(to_np(o.double()), h * c, tr.stored(h * c, 3 * EPS * np.abs(h * c), d), "scaled")

def test_norm_of_extreme_values():
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[norm extremes]")
    dev = "cuda"
    # squares far outside float32
    for v in (1e30, 1e-30, 3e38):
        g = [torch.full((10007,), v, device=dev)]
        want = float(np.float32(v)) * np.sqrt(10007.0)
        got = float(gs.grad_norm(g))
        assert got == np.inf if want > 3.41e38 else abs(got - want) <= 2 * EPS * want, v
    # empty tensors only, and no tensors of any size
    z = torch.zeros((0,), device=dev)
    assert float(gs.grad_norm([z])) == 0.0
    assert float(gs.clip_grads([z, z], 1.0)) == 0.0
    # zero gradients: norm 0, unchanged
    z = torch.zeros((5000,), device=dev)
    assert float(gs.clip_grads([z], 1.0)) == 0.0 and not z.any()
    # infinities and NaN: the norm tells, the factor is 0 or NaN
    for at in (0, 4096, 9999):
        g = torch.ones((10000,), device=dev)
        g[at] = float("inf")
        for kind in (gs.NORM_L2, gs.NORM_MAX):
            h = g.clone()
            assert float(gs.clip_grads([h], 1.0, kind)) == np.inf
            assert int(torch.isnan(h).sum()) == 1 and float(h.nan_to_num().abs().sum()) == 0.0
        g[at] = float("nan")
        for kind in (gs.NORM_L2, gs.NORM_MAX):
            h = g.clone()
            assert np.isnan(float(gs.clip_grads([h], 1.0, kind))) and torch.isnan(h).all()


def _adam_bounds(want, p, g, m, c, t, lr, b1, b2, eps, dtype):
    """What float32 may be off by from the float64 values `want` of (p, m, v): each constant, product and sum
    rounds once. m: two roundings on b1 m, four on (1 - b1) c g, one on the sum; v: the same with
    two more for the square; v is a sum of terms of one sign, so its error is relative (9 eps),
    and with the bias correction and the root the denominator's is below 8 eps."""
    p1, m1, v1 = want
    g = c * g
    Em = EPS * (2 * np.abs(b1 * m) + 5 * np.abs((1 - b1) * g) + np.abs(m1))
    Ev = EPS * 9 * v1
    i1, i2 = 1 / (1 - b1 ** t), 1 / (1 - b2 ** t)
    den = np.sqrt(v1 * i2) + eps
    q = m1 * i1 / den
    Eq = (Em * i1 + 2 * EPS * np.abs(m1 * i1)) / den + 9 * EPS * np.abs(q)
    Ep = 2 * EPS * np.abs(p) + lr * (Eq + EPS * np.abs(q)) + EPS * np.abs(p1)
    tiny = 2.0 ** -149  # subnormal products
    return tr.stored(p1, Ep, dtype), Em + tiny, Ev + tiny


@pytest.mark.parametrize("which", ["one", "few", "mlp", "edges", "many", "large"])
@pytest.mark.parametrize("pmix,gmix", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("mixed", "mixed"),
                                       ("f16", "f32")])
def test_adam_parity(which, pmix, gmix):
    import torch
    import gaussian_splatting_tile_amd as gs
    say(f"[adam {which} params {pmix} grads {gmix}]")
    sizes = LISTS[which]
    n = len(sizes)
    ptypes, gtypes = _types(pmix, n), _types(gmix, n)
    params = _grads(1, sizes, ptypes)
    grads = _grads(2, sizes, gtypes, 0.5)
    m, v = _grads(3, sizes, ["f32"] * n, 0.1), [x * x for x in _grads(4, sizes, ["f32"] * n, 0.2)]
    lr = [float(np.float32(1e-3 * (1 + k % 4))) for k in range(n)]
    wd = [float(np.float32(0.05 * (k % 3))) for k in range(n)]
    norm = tr.grad_norm([to_np(g.double()) for g in grads])
    for max_norm, start in ((0.0, 0), (float(np.float32(0.3 * norm)), 7), (float(np.float32(3 * norm)), 123456)):
        P, M, V = ([t.clone() for t in ts] for ts in (params, m, v))
        opt = gs.Adam(P, grads, lr=lr, weight_decay=wd, max_norm=max_norm, exp_avg=M, exp_avg_sq=V, step=start)
        got = opt.step()
        torch.cuda.synchronize()
        assert int(opt.steps) == start + 1
        assert (got is None) == (max_norm == 0.0)
        if got is not None:
            assert abs(float(got) - norm) <= norm * (EPS + sum(sizes) * 2.0 ** -53)
        c = tr.clip_factor(norm, max_norm) if max_norm else 1.0
        for k in range(n):
            args = [to_np(t[k].double()) for t in (params, grads, m, v)]
            with np.errstate(all="ignore"):
                want = tr.adam(*args, start, lr[k], wd[k], 0.9, 0.999, 1e-8, c)
                bounds = _adam_bounds(want, *args[:3], c, start + 1, lr[k], 0.9, 0.999, 1e-8, ptypes[k])
            for w, bound, t, name in zip(want, bounds, (P, M, V), ("param", "m", "v")):
                _close(to_np(t[k].double()), w, bound, (name, k, max_norm))


def test_adam_steps_and_skipped_steps():
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[adam skip]")
    for n in (100, 300000):
        p, g = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
        opt = gs.Adam([p], [g], lr=0.01, max_norm=1.0, skip_nonfinite=True)
        for k in range(3):
            opt.step()
        assert int(opt.steps) == 3
        was = [t.clone() for t in (p, opt.exp_avg[0], opt.exp_avg_sq[0])]
        for bad in (float("nan"), float("inf"), -float("inf")):
            g[n // 2] = bad
            norm = opt.step()
            torch.cuda.synchronize()
            assert not np.isfinite(float(norm)) and int(opt.steps) == 3
            for a, b in zip(was, (p, opt.exp_avg[0], opt.exp_avg_sq[0])):
                assert torch.equal(a, b)
        g[n // 2] = 0.0
        opt.step()
        assert int(opt.steps) == 4 and not torch.equal(was[0], p)


def test_adam_follows_changed_rates():
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[adam rates]")
    p = [torch.ones(10, device="cuda"), torch.ones(10, device="cuda")]
    g = [torch.ones(10, device="cuda"), torch.ones(10, device="cuda")]
    opt = gs.Adam(p, g, lr=[0.0, 0.5])
    opt.step()
    assert (p[0] == 1.0).all() and abs(float(p[1][0]) - 0.5) < 1e-6
    opt.set_lr([0.5, 0.0])
    opt.step()
    assert abs(float(p[0][0]) - 0.5) < 1e-6 and abs(float(p[1][0]) - 0.5) < 1e-6


def test_training_calls_are_deterministic_and_use_their_stream():
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[training deterministic]")
    sizes = [1_000_003, 17, 300_000]
    grads = _grads(5, sizes, ["f32", "bf16", "f16"])
    first, side = None, torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(4):
        with torch.cuda.stream(side):
            outs = [torch.empty_like(g) for g in grads]
            lst = gs.GradList(grads, out=outs)
            n = lst.clip(1.0)
            P = [torch.ones(s, device="cuda") for s in sizes]
            gs.Adam(P, grads, max_norm=1.0).step()
        torch.cuda.synchronize()
        if first is None:
            first = (n, outs, P)
        assert torch.equal(first[0], n)
        assert all(torch.equal(a, b) for a, b in zip(first[1] + first[2], outs + P))


def test_training_calls_on_a_given_stream():
    """A stream argument that is not the current stream, workspaces that the call allocates."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[training other stream]")
    side = torch.cuda.Stream()
    g = [torch.randn(100_000, device="cuda"), torch.randn(77, device="cuda")]
    x = torch.randn((1, 400, 70), device="cuda")
    want_n, want_h = gs.grad_norm(g), gs.recurrence_fwd(x, x, gating=gs.GATE_SIGMOID)["h"]
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        n = gs.grad_norm(g, stream=side)
        h = gs.recurrence_fwd(x, x, gating=gs.GATE_SIGMOID, stream=side)["h"]
        torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda")  # what the current stream allocates next
        side.synchronize()
        assert torch.equal(n, want_n) and torch.equal(h, want_h)


def test_training_calls_in_a_graph():
    """A recorded step counts its replays and follows its buffers."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[training graph]")
    sizes = [70000, 33, 4096]

    def make():
        return [torch.ones(s, device="cuda") for s in sizes], [torch.zeros(s, device="cuda") for s in sizes]

    p, g = make()
    q, h = make()
    a, b = gs.Adam(p, g, lr=0.01, max_norm=1.0), gs.Adam(q, h, lr=0.01, max_norm=1.0)
    clipped = [torch.empty_like(x) for x in g]
    lst = gs.GradList(g, out=clipped)
    norm = torch.zeros((), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lst.clip(1.0, out=norm)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lst.clip(1.0, out=norm)
        a.step()
    for k in range(4):
        for x, y in zip(g, h):
            x.copy_(torch.randn_like(x))
            y.copy_(x)
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        assert int(a.steps) == int(b.steps) == k + 1
        assert all(torch.equal(x, y) for x, y in zip(p + a.exp_avg + a.exp_avg_sq, q + b.exp_avg + b.exp_avg_sq))
        assert torch.equal(norm, b.norm)
        want = [torch.empty_like(x) for x in g]
        gs.GradList(h, out=want).clip(1.0)
        assert all(torch.equal(x, y) for x, y in zip(clipped, want))


def test_norm_past_32_bits():
    """2.2e9 elements of one tensor."""
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[norm 2.2e9 elements]")
    n = (1 << 31) + 12345
    g = torch.ones((n,), dtype=torch.bfloat16, device="cuda")
    g[-1] = 3.0
    norm = gs.clip_grads([g], 1.0)
    want = np.sqrt(n + 8.0)
    assert abs(float(norm) - want) <= 2 * EPS * want
    c = 1.0 / (want + 1e-6)
    assert abs(float(g[-1]) - 3 * c) <= 2.0 ** -7 * 3 * c and abs(float(g[-2]) - c) <= 2.0 ** -7 * c
    assert abs(float(g[0]) - c) <= 2.0 ** -7 * c


def test_training_calls_refuse():
    import torch
    import gaussian_splatting_tile_amd as gs
    say("[training refusals]")
    g = torch.zeros((8,), device="cuda")
    with pytest.raises(ValueError):
        gs.GradList([])
    with pytest.raises(TypeError):
        gs.GradList([g.double()])
    with pytest.raises(TypeError):
        gs.GradList([g.cpu()])
    with pytest.raises(ValueError):
        gs.GradList([torch.zeros((4, 4), device="cuda").t()[:2]])
    with pytest.raises(TypeError):
        gs.GradList([g], out=[g.bfloat16()])
    with pytest.raises(ValueError):
        gs.GradList([g], out=[g, g])
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(gs.GsError):
            gs.clip_grads([g], bad)
    with pytest.raises(gs.GsError):
        gs.grad_norm([g], kind=3)
    for kw in (dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=0.0), dict(max_norm=-1.0),
               dict(lr=float("nan")), dict(weight_decay=float("inf"))):
        with pytest.raises(gs.GsError):
            gs.Adam([g.clone()], [g], **kw).step()
    with pytest.raises(ValueError):
        gs.Adam([g], [torch.zeros((9,), device="cuda")])
    with pytest.raises(ValueError):
        gs.Adam([g], [g], step=-1)
    with pytest.raises(ValueError):
        gs.Adam([g], [g], lr=[1.0, 2.0])
    with pytest.raises(TypeError):
        gs.Adam([g], [g], exp_avg=[g.bfloat16()])
