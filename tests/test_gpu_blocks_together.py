"""A recurrent block as a model runs it: norm, one projection to queries, keys, values, gates, the delta rule, the heads'
gated norm, a projection back, residual and the next block's norm; forward, backward, and token by token."""
from __future__ import annotations

import numpy as np
import pytest

from gaussian_splatting_tile_amd._lib import GS_DELTA_FEW
from oracle import blocks

pytestmark = pytest.mark.gpu
B, HK, H, DK, DV, D = 2, 2, 4, 32, 48, 160
SIZES = [HK * DK, HK * DK, H * DV, H * DV]


def _type(dtype):
    import torch
    return dict(f32=torch.float32, bf16=torch.bfloat16)[dtype]


def make(T, dtype, seed):
    import torch
    rng = np.random.default_rng(seed)
    f = lambda *s: torch.tensor(rng.standard_normal(s).astype(np.float32), device="cuda")  # noqa: E731
    t = _type(dtype)
    return dict(x=f(B, T, D).to(t), w_in=(f(D, sum(SIZES)) / D ** 0.5).to(t), w_gates=f(D, 2 * H) / D ** 0.5,
                w_out=(f(H * DV, D) / (H * DV) ** 0.5).to(t), first=1 + 0.2 * f(D), heads=1 + 0.2 * f(DV),
                second=1 + 0.2 * f(D), scale=0.5 * f(D), h0=f(B, H, DK, DV), up=f(B, T, D).to(t), up_norm=f(B, T, D).to(t))


def split(rows):
    T = rows.shape[1]
    q, k, v, z = rows.split(SIZES, 2)  # parts of the projection's rows
    return q.unflatten(2, (HK, DK)), k.unflatten(2, (HK, DK)), v.unflatten(2, (H, DV)), z.unflatten(2, (H, DV)), T


def forward(m, h=None, out=None):
    """Every stage's inputs and outputs; x may be a part of the steps."""
    import torch
    import gaussian_splatting_tile_amd as gs
    x = m["x"]
    norm = gs.block_norm_fwd(x, pre=gs.BLOCK_NORM_RMS, pre_weight=m["first"])["norm"]
    q, k, v, z, T = split((norm.flatten(0, 1) @ m["w_in"]).view(B, -1, sum(SIZES)))
    q, k = q / 4, k / 4  # keys of a length near 1
    gates = (norm.flatten(0, 1).float() @ m["w_gates"]).view(B, T, 2 * H)
    log_decay, beta = -torch.nn.functional.softplus(gates[..., :H]), torch.sigmoid(gates[..., H:])
    d = dict(q=q, k=k, v=v, log_decay=log_decay, beta=beta, h0=m["h0"] if h is None else h)
    s = gs.delta_rule_fwd(**d, checkpoints=h is None, out=out)
    heads = dict(y=s["o"], gate=z, post_weight=m["heads"])
    y = gs.block_norm_fwd(**heads, gating=gs.BLOCK_GATE_SILU, post=gs.BLOCK_NORM_RMS)["out"]
    back = dict(y=(y.flatten(0, 1).flatten(1) @ m["w_out"]).view(B, T, D), residual=x, scale=m["scale"], pre_weight=m["second"])
    last = gs.block_norm_fwd(**back, pre=gs.BLOCK_NORM_RMS)
    return dict(norm=norm, d=d, s=s, heads=heads, y=y, back=back, last=last)


def backward(m, f):
    """The gradients of every stage from those of the stage behind it."""
    import gaussian_splatting_tile_amd as gs
    last = gs.block_norm_bwd(**f["back"], grad_out=m["up"], grad_norm=m["up_norm"], pre=gs.BLOCK_NORM_RMS)
    gy = (last["grad_y"].flatten(0, 1) @ m["w_out"].t()).view(f["y"].shape)
    heads = gs.block_norm_bwd(**f["heads"], grad_out=gy, gating=gs.BLOCK_GATE_SILU, post=gs.BLOCK_NORM_RMS)
    delta = gs.delta_rule_bwd(**f["d"], ckpt=f["s"]["ckpt"], grad_o=heads["grad_y"])
    return dict(last=last, gy=gy, heads=heads, delta=delta)


def host(d):
    import torch
    return {k: v.double().cpu().numpy() for k, v in d.items() if isinstance(v, torch.Tensor)}


def close(out, want, dtype, f32=(), lost=None):
    for name in want:
        if name in ("sizes", "terms") or out.get(name) is None:
            continue
        g = out[name]
        kind = "f32" if g.dim() == 1 or name in f32 else dtype
        far = blocks.off(g.double().cpu().numpy(), want[name], kind, 2.0 if g.dim() == 1 else 1.0,
                         want.get("sizes", {}).get(name, 0.0), **({"lost": lost} if name == "o" and lost is not None else {}))
        assert far <= 1, (name, far)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 70, 200])
def test_every_stage(T, dtype):
    """Each stage against the oracle on the inputs that it had, so no error of the stages in front counts."""
    m = make(T, dtype, T)
    f = forward(m)
    g = backward(m, f)
    up = dict(grad_out=m["up"], grad_norm=m["up_norm"])
    close(dict(f["last"], **g["last"]), blocks.block_norm(**host(f["back"]), **host(up), pre="rms", eps=1e-6), dtype)
    close(dict(out=f["y"], **g["heads"]), blocks.block_norm(**host(f["heads"]), grad_out=host(dict(g=g["gy"]))["g"],
                                                            gating="silu", post="rms", eps=1e-6), dtype)
    want = blocks.delta_rule(**host(f["d"]), grad_o=host(dict(g=g["heads"]["grad_y"]))["g"], terms=True)
    chunked = dtype == "bf16" and T > GS_DELTA_FEW
    close(dict(o=f["s"]["o"], h_last=f["s"]["h_last"], **g["delta"]), want, dtype,
          ("h_last", "grad_h0", "grad_log_decay", "grad_beta"), blocks.LOST * want["terms"] if chunked else None)


def test_captured_block():
    """The whole block, forward and backward, in one graph: replays on new inputs equal eager runs, bit for bit."""
    import torch
    m, new = make(130, "bf16", 1), make(130, "bf16", 2)

    def run(m):
        f = forward(m)
        g = backward(m, f)
        return dict(**f["last"], h_last=f["s"]["h_last"], **{"d_" + k: v for k, v in g["delta"].items()},
                    **{"l_" + k: v for k, v in g["last"].items()}, **{"h_" + k: v for k, v in g["heads"].items()})

    want, other = run(m), run(new)
    buf = {k: v.clone() for k, v in m.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(buf)
    for src, ref in ((new, other), (m, want), (new, other)):
        for k in buf:
            buf[k].copy_(src[k])
        graph.replay()
        torch.cuda.synchronize()
        for k in got:
            assert got[k] is None or torch.equal(got[k], ref[k]), k
        run(m)


def test_prompt_and_tokens():
    """A prompt in one call and then token by token, in one state buffer, is the sequence in one call. In float32, where
    both are off by the oracle's TOL of a sum's size: the states and outputs of the two ways by twice that."""
    import torch
    import gaussian_splatting_tile_amd as gs
    m = make(90, "f32", 7)
    whole = forward(m)
    h, outs = m["h0"].clone(), []
    for a, b in [(0, 70)] + [(t, t + 1) for t in range(70, 86)] + [(86, 90)]:
        part = dict(m, x=m["x"][:, a:b])
        d = {k: v[:, a:b] if k != "h0" else h for k, v in whole["d"].items()}
        s = gs.delta_rule_fwd(**d, out=dict(h_last=h))
        assert s["h_last"] is h
        outs.append(s["o"])
        assert torch.equal(forward(part, m["h0"])["norm"], whole["norm"][:, a:b])  # rows do not depend on their neighbours
    want = blocks.delta_rule(**host(whole["d"]))
    assert blocks.off(torch.cat(outs, 1).double().cpu().numpy(), want["o"]) <= 1
    assert blocks.off(h.double().cpu().numpy(), want["h_last"]) <= 1
    assert blocks.off(whole["s"]["h_last"].double().cpu().numpy(), want["h_last"]) <= 1


def test_two_streams_at_once():
    """Two calls of every operator at the same time, each with its own workspace, many times over."""
    import torch
    import gaussian_splatting_tile_amd as gs
    ms = [make(300, "bf16", 11), make(300, "bf16", 12)]
    want = [(forward(m), None) for m in ms]
    want = [(f, backward(m, f)) for m, (f, _) in zip(ms, want)]
    n = gs.delta_rule_scratch_bytes(B, 300, H, DK, DV, True, torch.bfloat16, key_heads=HK)
    scratch = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in ms]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for (f, g), s, ws in zip(want, streams, scratch):
            out = gs.delta_rule_fwd(**f["d"], checkpoints=True, stream=s)
            back = gs.delta_rule_bwd(**f["d"], ckpt=out["ckpt"], grad_o=g["heads"]["grad_y"], scratch=ws, stream=s)
            heads = gs.block_norm_bwd(**f["heads"], grad_out=g["gy"], gating=gs.BLOCK_GATE_SILU, post=gs.BLOCK_NORM_RMS, stream=s)
            got.append((out, back, heads))
        torch.cuda.synchronize()
        for (out, back, heads), (f, g) in zip(got, want):
            assert torch.equal(out["o"], f["s"]["o"]) and torch.equal(out["h_last"], f["s"]["h_last"])
            for k in back:
                assert torch.equal(back[k], g["delta"][k]), k
            for k in heads:
                assert heads[k] is None or torch.equal(heads[k], g["heads"][k]), k
