"""The gated delta rule on the GPU against the float64 oracle, step by step, at the sizes and masks where chunks,
tiles and short calls can go wrong."""
from __future__ import annotations

import numpy as np
import pytest

from gaussian_splatting_tile_amd._lib import GS_DELTA_FEW
from oracle import blocks

pytestmark = pytest.mark.gpu
TYPES = ("f32", "bf16", "f16")


def _torch_type(dtype):
    import torch
    return dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[dtype]


def make(B, T, Hk, H, dk, dv, dtype, seed, ragged=False, restarts=False, packed=False, train=True, state=True):
    """Inputs on the GPU as the operator takes them, and the same as float64 arrays."""
    import torch
    rng = np.random.default_rng(seed)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    unit = lambda x: x / (np.linalg.norm(x, axis=-1, keepdims=True) + 1e-6)  # noqa: E731
    t = _torch_type(dtype)
    q, k, v = unit(np.abs(f(B, T, Hk, dk)) - 0.3), unit(np.abs(f(B, T, Hk, dk)) - 0.3), f(B, T, H, dv)
    if packed:
        rows = torch.tensor(np.concatenate([x.reshape(B, T, -1) for x in (q, k, v)], 2), device="cuda").to(t)
        parts = rows.split([Hk * dk, Hk * dk, H * dv], 2)
        d = dict(q=parts[0].unflatten(2, (Hk, dk)), k=parts[1].unflatten(2, (Hk, dk)), v=parts[2].unflatten(2, (H, dv)))
    else:
        d = {n: torch.tensor(x, device="cuda").to(t) for n, x in (("q", q), ("k", k), ("v", v))}
    d["log_decay"] = torch.tensor(-np.exp(f(B, T, H) + 1.5 * f(H) - 3), device="cuda")
    d["beta"] = torch.tensor((1 / (1 + np.exp(-f(B, T, H)))).astype(np.float32), device="cuda")
    if state:
        d["h0"] = torch.tensor(f(B, H, dk, dv), device="cuda")
    if ragged:
        lengths = rng.integers(0, T + 1, B).astype(np.int32)
        lengths[0] = T
        if B > 2:
            lengths[1:3] = 0, 1
        d["lengths"] = torch.tensor(lengths, device="cuda")
    if restarts:
        d["restart"] = torch.tensor((rng.random((B, T)) < 6.0 / (T + 6)).astype(np.uint8), device="cuda")
    up = dict(grad_o=torch.tensor(f(B, T, H, dv), device="cuda").to(t),
              grad_last=torch.tensor(f(B, H, dk, dv), device="cuda")) if train else {}
    return d, up


def host(d):
    import torch
    return {k: v.double().cpu().numpy() if v.is_floating_point() else v.cpu().numpy() for k, v in d.items()
            if isinstance(v, torch.Tensor)}


def run(d, up, scale=None):
    import gaussian_splatting_tile_amd as gs
    out = gs.delta_rule_fwd(**d, scale=scale, checkpoints=bool(up))
    if up:
        out.update(gs.delta_rule_bwd(**d, scale=scale, ckpt=out["ckpt"], **up))
    return out


def check(out, want, dtype, sums=1.0):
    for name, w in want.items():
        if name == "terms":
            continue
        kind = "f32" if name in ("h_last", "grad_h0", "grad_log_decay", "grad_beta") else dtype
        # LOST is derived for the kernels that work in chunks, which take what is more than a few steps
        chunked = w.shape[1] > GS_DELTA_FEW
        lost = blocks.LOST * want["terms"] if name == "o" and dtype == "bf16" and chunked else 0.0
        far = blocks.off(out[name].double().cpu().numpy(), w, kind, sums, lost=lost)
        assert far <= 1, (name, far)


# B, T, Hk, H, dk, dv, flags
CASES = [
    (1, 1, 1, 1, 16, 16, ""), (2, 1, 2, 4, 128, 128, "p"), (3, 2, 1, 3, 17, 33, ""), (2, 5, 2, 2, 64, 64, "r"),
    (3, 8, 2, 4, 128, 100, "lr"), (3, 9, 2, 4, 128, 100, "lr"), (2, 100, 2, 6, 128, 128, "p"),
    (2, 150, 1, 5, 48, 40, "lr"), (1, 70, 1, 9, 128, 32, ""),
    (1, 15, 1, 1, 1, 1, ""), (2, 16, 1, 2, 8, 128, "p"), (1, 17, 2, 2, 128, 8, ""), (2, 63, 1, 1, 40, 24, "r"),
    (1, 64, 2, 4, 64, 64, "p"), (1, 65, 1, 2, 64, 128, "r"), (4, 130, 2, 2, 128, 64, "lr"), (3, 200, 2, 6, 24, 40, "lrp"),
    (1, 257, 1, 1, 100, 128, "p"), (2, 192, 2, 4, 128, 128, "lr"), (5, 129, 1, 2, 72, 56, "l"),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,T,Hk,H,dk,dv,flags", CASES)
def test_against_oracle(B, T, Hk, H, dk, dv, flags, dtype):
    d, up = make(B, T, Hk, H, dk, dv, dtype, 7 * T + dk, "l" in flags, "r" in flags, "p" in flags)
    out = run(d, up)
    check(out, blocks.delta_rule(**host(d), **host(up), terms=True), dtype)
    again = run(d, up)
    for k in out:
        if out[k] is not None and k != "ckpt":
            assert (out[k] == again[k]).all(), k


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,T,Hk,H,dk,dv,flags", [
    (1, 2048, 1, 1, 64, 64, ""), (1, 2100, 1, 2, 128, 128, "p"), (2, 2500, 1, 1, 40, 72, "lr"), (3, 2049, 1, 1, 100, 16, "l"),
])
def test_long_sequences(B, T, Hk, H, dk, dv, flags, dtype):
    """Few sequences of many chunks: cut into segments that run side by side."""
    d, up = make(B, T, Hk, H, dk, dv, dtype, T + dk, "l" in flags, "r" in flags, "p" in flags)
    h = d["h0"].clone()
    out = run(d, up)
    check(out, blocks.delta_rule(**host(d), **host(up), terms=True), dtype)
    import gaussian_splatting_tile_amd as gs
    again = gs.delta_rule_fwd(**dict(d, h0=h), out=dict(h_last=h))
    assert (h == out["h_last"]).all() and (again["o"] == out["o"]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 3, 70])
def test_without_state_and_upstream_state(T, dtype):
    d, up = make(2, T, 2, 2, 64, 32, dtype, 5, state=False)
    del up["grad_last"]
    check(run(d, up, scale=0.7), blocks.delta_rule(**host(d), **host(up), scale=0.7, terms=True), dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_hard_gates(dtype):
    """Decays of 0 (a drop), of almost 0 and of exactly 1, beta of 0 and 1, and one key all along."""
    import torch
    d, up = make(2, 150, 1, 2, 32, 48, dtype, 11)
    d["k"] = d["k"][:, :1].expand(-1, 150, -1, -1)
    g = d["log_decay"]
    g[:, ::3] = 0.0
    g[:, 40] = -float("inf")
    g[:, 41] = -200.0
    g[:, 70:90:4] = -60.0
    g[:, 100] = -104.5
    d["beta"][:, ::2], d["beta"][:, 1::4] = 1.0, 0.0
    out, want = run(d, up), blocks.delta_rule(**host(d), **host(up), terms=True)
    assert torch.isfinite(out["grad_log_decay"]).all()
    # a key that is stored again and again cancels what the chunk's sums hold: 64 terms that leave one
    check(out, want, dtype, 8.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_nothing_of_padding_is_read(dtype):
    import torch
    nan = float("nan")
    d, up = make(3, 140, 2, 2, 64, 64, dtype, 13, ragged=True)
    want = run(d, up)
    dirty = {k: v.clone() for k, v in d.items()}
    dup = {k: v.clone() for k, v in up.items()}
    for b in range(3):
        n = int(d["lengths"][b])
        for k in ("q", "k", "v", "log_decay", "beta"):
            dirty[k][b, n:] = nan
        dup["grad_o"][b, n:] = nan
    got = run(dirty, dup)
    for k in want:
        if k != "ckpt":
            assert torch.equal(got[k], want[k]), k
    for b in range(3):
        n = int(d["lengths"][b])
        for k in ("o", "grad_q", "grad_k", "grad_v", "grad_log_decay", "grad_beta"):
            assert (got[k][b, n:] == 0).all(), k
    assert torch.equal(got["h_last"][1], d["h0"][1]) and torch.equal(got["grad_h0"][1], up["grad_last"][1])


@pytest.mark.parametrize("T", [1, 4, 100])
def test_state_in_place_and_buffers(T):
    """h_last replaces h0; given outputs and workspace are used; rows of the caller's around them stay."""
    import torch
    import gaussian_splatting_tile_amd as gs
    d, _ = make(2, T, 1, 2, 64, 80, "bf16", 17, train=False)
    want = gs.delta_rule_fwd(**d)
    around = torch.full((4, T, 2, 80), 7.0, device="cuda", dtype=torch.bfloat16)
    h = d["h0"].clone()
    n = gs.delta_rule_scratch_bytes(2, T, 2, 64, 80, dtype=torch.bfloat16)
    scratch = torch.full((n + 64,), 171, dtype=torch.uint8, device="cuda")
    out = gs.delta_rule_fwd(**dict(d, h0=h), out=dict(o=around[1:3], h_last=h), scratch=scratch[:n])
    assert out["h_last"] is h and torch.equal(h, want["h_last"]) and torch.equal(around[1:3], want["o"])
    assert (around[0] == 7).all() and (around[3] == 7).all() and (scratch[n:] == 171).all()


def test_steps_one_by_one_equal_one_call():
    import gaussian_splatting_tile_amd as gs
    d, _ = make(2, 150, 2, 4, 64, 64, "f32", 19, restarts=True, train=False)
    whole = gs.delta_rule_fwd(**d)
    want = blocks.delta_rule(**host(d))
    h, at = d["h0"].clone(), 0
    for n in (1, 2, 1, 5, 16, 64, 1, 33, 27):
        part = {k: v[:, at:at + n] if k != "h0" else h for k, v in d.items()}
        part["restart"] = part["restart"].contiguous()
        o = gs.delta_rule_fwd(**part, out=dict(h_last=h))["o"]
        assert blocks.off(o.cpu().numpy(), want["o"][:, at:at + n]) <= 1, n
        at += n
    assert at == 150
    assert blocks.off(h.cpu().numpy(), want["h_last"]) <= 1
    assert blocks.off(whole["h_last"].cpu().numpy(), want["h_last"]) <= 1


def test_strides_of_zero_and_of_heads():
    """A value repeated over the batch, heads in front of steps, and gates that are a part of wider rows."""
    import torch
    d, up = make(2, 90, 2, 2, 32, 32, "bf16", 23)
    e = dict(d)
    e["v"] = d["v"][:1].expand(2, -1, -1, -1)
    e["q"] = d["q"].transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.cat([d["beta"], d["log_decay"]], 2)
    e["beta"], e["log_decay"] = wide[..., :2], wide[..., 2:]
    check(run(e, up), blocks.delta_rule(**host(e), **host(up), terms=True), "bf16")


def test_unaligned_rows():
    import torch
    d, up = make(2, 80, 1, 1, 64, 64, "bf16", 29)
    e = dict(d)
    for k in ("q", "k", "v"):
        flat = torch.empty(d[k].numel() + 1, device="cuda", dtype=d[k].dtype)
        e[k] = flat[1:].view(d[k].shape)
        e[k].copy_(d[k])
    check(run(e, up), blocks.delta_rule(**host(d), **host(up), terms=True), "bf16")


@pytest.mark.parametrize("T", [1, 150])
def test_streams_and_graph(T):
    """Another stream, and a captured forward and backward replayed on new inputs between eager calls."""
    import torch
    import gaussian_splatting_tile_amd as gs
    d, up = make(2, T, 1, 2, 64, 64, "bf16", 31, restarts=True)
    new, up2 = make(2, T, 1, 2, 64, 64, "bf16", 37, restarts=True)
    want, other = run(d, up), run(new, up2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = gs.delta_rule_fwd(**d, checkpoints=True, stream=side)
    back = gs.delta_rule_bwd(**d, ckpt=out["ckpt"], **up, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for k in ("o", "h_last"):
        assert torch.equal(out[k], want[k])
    for k in back:
        assert torch.equal(back[k], want[k]), k
    buf, bup = {k: v.clone() for k, v in d.items()}, {k: v.clone() for k, v in up.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(buf, bup)
    for src, sup, ref in ((new, up2, other), (d, up, want), (new, up2, other)):
        for k in buf:
            buf[k].copy_(src[k])
        for k in bup:
            bup[k].copy_(sup[k])
        graph.replay()
        torch.cuda.synchronize()
        for k in got:
            if k != "ckpt" and got[k] is not None:
                assert torch.equal(got[k], ref[k]), k
        run(d, up)


def test_empty():
    import torch
    import gaussian_splatting_tile_amd as gs
    e = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    h = torch.randn((2, 2, 8, 8), device="cuda")
    out = gs.delta_rule_fwd(e(2, 0, 1, 8), e(2, 0, 1, 8), e(2, 0, 2, 8), e(2, 0, 2), e(2, 0, 2), h0=h)
    assert out["o"].shape == (2, 0, 2, 8) and torch.equal(out["h_last"], h)
    back = gs.delta_rule_bwd(e(2, 0, 1, 8), e(2, 0, 1, 8), e(2, 0, 2, 8), e(2, 0, 2), e(2, 0, 2), e(2, 0, 2, 8), h0=h,
                             grad_last=h)
    assert torch.equal(back["grad_h0"], h)
    assert gs.delta_rule_fwd(e(0, 3, 1, 8), e(0, 3, 1, 8), e(0, 3, 2, 8), e(0, 3, 2), e(0, 3, 2))["o"].shape == (0, 3, 2, 8)


@pytest.mark.parametrize("T", [5, 70])
def test_offsets_past_32_bits(T):
    """Sequences and heads that lie more than 2^31 elements apart in one buffer."""
    import torch
    d, up = make(2, T, 1, 2, 32, 48, "bf16", 47)
    far = 1 << 31
    buffer = torch.empty(2 * far + (1 << 16), dtype=torch.bfloat16, device="cuda")
    e = dict(d)
    for i, (k, by) in enumerate((("q", "batch"), ("k", "batch"), ("v", "head"))):
        B, _, H, dim = d[k].shape
        strides = (far, H * dim, dim, 1) if by == "batch" else (T * dim, dim, far, 1)
        e[k] = buffer.as_strided(d[k].shape, strides, i << 14)
        e[k].copy_(d[k])
    got, want = run(e, up), run(d, up)
    for k in want:
        if k != "ckpt":
            assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_state_in_place_in_segments(dtype):
    """h_last in h0's place where a sequence is cut into segments, forward; and the backward from that state."""
    import torch
    import gaussian_splatting_tile_amd as gs
    d, up = make(1, 2300, 1, 2, 64, 48, dtype, 53)
    want = run(d, up)
    h = d["h0"].clone()
    out = gs.delta_rule_fwd(**dict(d, h0=h), out=dict(h_last=h), checkpoints=True)
    assert torch.equal(h, want["h_last"]) and torch.equal(out["o"], want["o"])
    back = gs.delta_rule_bwd(**d, ckpt=out["ckpt"], **up)
    for k in back:
        assert torch.equal(back[k], want[k]), k
