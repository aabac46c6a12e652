"""The norms around a block on the GPU against the float64 oracle."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import blocks

pytestmark = pytest.mark.gpu
TYPES = ("f32", "bf16", "f16")


def _torch_type(dtype):
    import torch
    return dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[dtype]


def make(shape, dtype, seed, post, gating, pre, residual=True, scale=True, bias=True, packed=False, weight_type="f32"):
    import torch
    rng = np.random.default_rng(seed)
    t, wt, D = _torch_type(dtype), _torch_type(weight_type), shape[-1]
    f = lambda *s: torch.tensor(rng.standard_normal(s).astype(np.float32), device="cuda")  # noqa: E731
    d = dict(y=f(*shape) * (1 + f(*shape[:-1], 1).abs()) + 0.5, gate=f(*shape))
    if packed:  # parts of one projection's rows
        rows = torch.cat([x.reshape(shape[0], -1) for x in d.values()], 1).to(t)
        half = rows.shape[1] // 2
        d = dict(y=rows[:, :half].view(shape), gate=rows[:, half:].view(shape))
    else:
        d = {k: v.to(t) for k, v in d.items()}
    if gating == "none":
        del d["gate"]
    if residual:
        d["residual"] = (2 * f(*shape)).to(t)
    if scale:
        d["scale"] = (0.5 * f(D)).to(wt)
    if post != "none":
        d["post_weight"] = (1 + 0.2 * f(D)).to(wt)
        if bias:
            d["post_bias"] = f(D).to(wt)
    if pre != "none":
        d["pre_weight"] = (1 + 0.2 * f(D)).to(wt)
        if bias:
            d["pre_bias"] = f(D).to(wt)
    up = dict(grad_out=f(*shape).to(t), grad_norm=f(*shape).to(t) if pre != "none" else None)
    return d, up


def kinds(post, gating, pre):
    import gaussian_splatting_tile_amd as gs
    n = dict(none=gs.BLOCK_NORM_NONE, rms=gs.BLOCK_NORM_RMS, layer=gs.BLOCK_NORM_LAYER)
    g = dict(none=gs.BLOCK_GATE_NONE, sigmoid=gs.BLOCK_GATE_SIGMOID, silu=gs.BLOCK_GATE_SILU)
    return dict(post=n[post], gating=g[gating], pre=n[pre])


def run(d, up, post, gating, pre, eps, **kw):
    import gaussian_splatting_tile_amd as gs
    out = gs.block_norm_fwd(**d, **kinds(post, gating, pre), eps=eps)
    out.update(gs.block_norm_bwd(**d, **up, **kinds(post, gating, pre), eps=eps, **kw))
    return out


def host(d):
    return {k: v.double().cpu().numpy() for k, v in d.items() if v is not None}


def check(out, want, dtype, rows):
    # a sum over the rows adds up to 64 of a workgroup's one by one, then the workgroups'
    sums = max(1.0, (rows / 192.0) ** 0.5)
    for name, g in out.items():
        if g is None:
            continue
        whole = name.startswith("grad_") and g.dim() == 1
        far = blocks.off(g.double().cpu().numpy(), want[name], "f32" if whole else dtype, sums if whole else 1.0,
                         want["sizes"].get(name, 0.0))
        assert far <= 1, (name, far)


CASES = [
    ((1, 1), "rms", "silu", "rms"), ((3, 7), "layer", "sigmoid", "layer"), ((5, 64), "none", "none", "rms"),
    ((33, 77), "layer", "silu", "rms"), ((300, 128), "rms", "silu", "none"), ((17, 255), "rms", "none", "layer"),
    ((64, 512), "none", "sigmoid", "layer"), ((2, 2048), "rms", "sigmoid", "rms"), ((700, 1000), "layer", "silu", "layer"),
    ((9, 4096), "rms", "none", "rms"), ((3, 8192), "layer", "silu", "layer"), ((4, 8200), "rms", "sigmoid", "rms"),
    ((2, 16384), "layer", "silu", "rms"), ((2, 16383), "rms", "silu", "layer"), ((2500, 40), "rms", "silu", "rms"),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,post,gating,pre", CASES)
def test_against_oracle(shape, post, gating, pre, dtype):
    d, up = make(shape, dtype, sum(shape), post, gating, pre)
    out = run(d, up, post, gating, pre, 1e-5)
    want = blocks.block_norm(**host(d), **host(up), post=post, gating=gating, pre=pre, eps=1e-5)
    check(out, want, dtype, shape[0])
    again = run(d, up, post, gating, pre, 1e-5)
    for k in out:
        assert out[k] is None or (out[k] == again[k]).all(), k


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("residual,scale,bias", [(False, False, False), (True, False, False), (False, True, True)])
def test_parts_left_out(residual, scale, bias, dtype):
    shape = (40, 96)
    d, up = make(shape, dtype, 5, "rms", "silu", "rms", residual, scale, bias, weight_type=dtype)
    out = run(d, up, "rms", "silu", "rms", 1e-6)
    assert (out["grad_residual"] is None) == (not residual) and (out["grad_scale"] is None) == (not scale)
    assert (out["grad_pre_bias"] is None) == (not bias)
    check(out, blocks.block_norm(**host(d), **host(up), post="rms", gating="silu", pre="rms", eps=1e-6), dtype, 40)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(30, 4, 64), (11, 3, 50), (6, 2, 3, 24)])
def test_heads_of_a_projection(shape, dtype):
    d, up = make(shape, dtype, 3, "rms", "silu", "none", False, False, False, packed=True)
    out = run(d, up, "rms", "silu", "none", 1e-6)
    check(out, blocks.block_norm(**host(d), **host(up), post="rms", gating="silu", eps=1e-6), dtype, out["out"].numel())


def test_unaligned_rows():
    import torch
    d, up = make((50, 128), "bf16", 9, "rms", "silu", "rms")
    e = dict(d)
    flat = torch.empty(d["y"].numel() + 1, device="cuda", dtype=torch.bfloat16)
    e["y"] = flat[1:].view(50, 128)
    e["y"].copy_(d["y"])
    check(run(e, up, "rms", "silu", "rms", 1e-6),
          blocks.block_norm(**host(d), **host(up), post="rms", gating="silu", pre="rms"), "bf16", 50)


def test_broadcast_gate_and_only_the_norm():
    """One gate for all rows (stride 0); a norm whose sum is not wanted, and its gradient without the stream's."""
    import gaussian_splatting_tile_amd as gs
    d, up = make((60, 72), "f32", 15, "rms", "sigmoid", "rms")
    d["gate"] = d["gate"][:1].expand(60, -1)
    a = dict(**d, **kinds("rms", "sigmoid", "rms"))
    out = gs.block_norm_fwd(**a, want_out=False)
    assert out["out"] is None
    back = gs.block_norm_bwd(**a, grad_out=None, grad_norm=up["grad_norm"])
    want = blocks.block_norm(**host(d), grad_norm=host(up)["grad_norm"], post="rms", gating="sigmoid", pre="rms")
    check(dict(back, norm=out["norm"]), want, "f32", 60)


@pytest.mark.parametrize("shape", [(20, 64), (7, 100), (3, 5000)])
def test_in_place(shape):
    """out may replace y, gate or residual; gradients may replace those they come from."""
    import torch
    import gaussian_splatting_tile_amd as gs
    d, up = make(shape, "bf16", 21, "rms", "silu", "rms")
    k = kinds("rms", "silu", "rms")
    want = gs.block_norm_fwd(**d, **k)
    for name in ("y", "gate", "residual"):
        e = dict(d, **{name: d[name].clone()})
        got = gs.block_norm_fwd(**e, **k, out=dict(out=e[name]))
        assert got["out"] is e[name]
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["norm"], want["norm"])
    wb = gs.block_norm_bwd(**d, **up, **k)
    u = {n: x.clone() for n, x in up.items()}
    out = {n: None if x is None else torch.empty_like(x) for n, x in wb.items()}
    out.update(grad_y=u["grad_out"], grad_residual=u["grad_norm"])
    gs.block_norm_bwd(**d, **u, **k, out=out)
    for n in wb:
        assert torch.equal(out[n], wb[n]), n


def test_hard_rows():
    """Rows of zeros, of one value, of huge and of tiny elements; gates far from 0; a row that is not finite stays its own."""
    import torch
    import gaussian_splatting_tile_amd as gs
    d, up = make((8, 200), "f32", 25, "layer", "silu", "layer")
    d["y"][0], d["residual"][0] = 0.0, 0.0
    d["y"][1] = 5.0
    d["y"][2] *= 1e15
    d["y"][3] *= 1e-20
    d["gate"][4], d["gate"][5] = 100.0, -100.0
    k = kinds("layer", "silu", "layer")
    out = run(d, up, "layer", "silu", "layer", 1e-5)
    want = blocks.block_norm(**host(d), **host(up), post="layer", gating="silu", pre="layer", eps=1e-5)
    for r in range(8):
        for n in ("out", "norm", "grad_y", "grad_gate", "grad_residual"):
            if r == 1 and n == "grad_y":
                continue  # (y - mean) / sqrt(eps) of a mean that is rounded
            # sigma(-100) = 2^-144 is 1 / (1 + inf) = 0 in float32; nothing here multiplies it by more than 2^24
            assert blocks.off(out[n][r].cpu().numpy(), want[n][r], "f32", 8.0, lost=2.0 ** -120) <= 1, (r, n)
    clean = gs.block_norm_fwd(**d, **k, eps=1e-5)
    d["y"][6] = float("nan")
    dirty = gs.block_norm_fwd(**d, **k, eps=1e-5)
    for r in (0, 1, 2, 3, 4, 5, 7):
        assert torch.equal(dirty["norm"][r], clean["norm"][r])
    assert torch.isnan(dirty["norm"][6]).all()


def test_streams_and_graph():
    import torch
    import gaussian_splatting_tile_amd as gs
    d, up = make((600, 512), "bf16", 31, "rms", "silu", "rms")
    new, up2 = make((600, 512), "bf16", 33, "rms", "silu", "rms")
    k = kinds("rms", "silu", "rms")
    want, other = run(d, up, "rms", "silu", "rms", 1e-6), run(new, up2, "rms", "silu", "rms", 1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = gs.block_norm_fwd(**d, **k, stream=side)
    out.update(gs.block_norm_bwd(**d, **up, **k, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    for n in want:
        assert torch.equal(out[n], want[n]), n
    buf, bup = {n: v.clone() for n, v in d.items()}, {n: v.clone() for n, v in up.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(buf, bup, "rms", "silu", "rms", 1e-6)
    for src, sup, ref in ((new, up2, other), (d, up, want), (new, up2, other)):
        for n in buf:
            buf[n].copy_(src[n])
        for n in bup:
            bup[n].copy_(sup[n])
        graph.replay()
        torch.cuda.synchronize()
        for n in ref:
            assert torch.equal(got[n], ref[n]), n
        run(d, up, "rms", "silu", "rms", 1e-6)


def test_no_rows():
    import torch
    import gaussian_splatting_tile_amd as gs
    y, w = torch.zeros((0, 16), device="cuda"), torch.ones(16, device="cuda")
    k = kinds("rms", "none", "rms")
    assert gs.block_norm_fwd(y, post_weight=w, pre_weight=w, **k)["norm"].shape == (0, 16)
    back = gs.block_norm_bwd(y, y, grad_norm=y, post_weight=w, pre_weight=w, **k)
    assert (back["grad_post_weight"] == 0).all() and (back["grad_pre_weight"] == 0).all()


@pytest.mark.parametrize("post,gating,pre", [("rms", "none", "none"), ("layer", "silu", "layer"), ("rms", "silu", "rms")])
def test_rows_behind_the_last_with_no_eps(post, gating, pre):
    """A workgroup's threads that have no row add nothing to the sums, also where eps is 0 and a row of zeros has no norm."""
    for rows in (3, 33):
        d, up = make((rows, 64), "f32", 41, post, gating, pre)
        out = run(d, up, post, gating, pre, 0.0)
        want = blocks.block_norm(**host(d), **host(up), post=post, gating=gating, pre=pre, eps=0.0)
        check(out, want, "f32", rows)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("post,gating,pre", [("rms", "silu", "rms"), ("rms", "none", "rms"), ("rms", "sigmoid", "none"),
                                             ("none", "none", "rms"), ("layer", "sigmoid", "layer")])
@pytest.mark.parametrize("shape", [(1700, 500), (1100, 2048), (530, 2050), (520, 4100), (300, 9000)])
def test_more_rows_than_workgroups(shape, post, gating, pre, bias, dtype):
    """Every kind of backward kernel at every width, with rows that a workgroup takes one after another."""
    d, up = make(shape, dtype, 43, post, gating, pre, bias=bias)
    out = run(d, up, post, gating, pre, 1e-5)
    check(out, blocks.block_norm(**host(d), **host(up), post=post, gating=gating, pre=pre, eps=1e-5), dtype, shape[0])


def test_offsets_past_32_bits():
    """Rows that lie more than 2^31 elements apart in one buffer."""
    import torch
    d, up = make((3, 64), "bf16", 47, "rms", "silu", "rms")
    far = 1 << 31
    buffer = torch.empty(2 * far + 4096, dtype=torch.bfloat16, device="cuda")
    e = dict(d)
    for i, k in enumerate(("y", "gate", "residual")):
        e[k] = buffer.as_strided((3, 64), (far, 1), i * 1024 + i)
        e[k].copy_(d[k])
    got, want = run(e, up, "rms", "silu", "rms", 1e-6), run(d, up, "rms", "silu", "rms", 1e-6)
    for k in want:
        assert want[k] is None or torch.equal(got[k], want[k]), k
