"""The example that runs the recurrence, the appearance MLP, the rasterizer, the clipping and
Adam together: its gradient against the oracles' chain, and a fit that gets better."""
import importlib.util
import os
import sys

import numpy as np
import pytest

from gpu_helpers import GRAD_REL, to_np
from oracle import appearance as app
from oracle import training as tr

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("fit_clip", os.path.join(ROOT, "examples", "fit_clip.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_clip_gradient_matches_the_oracle_chain(example, orc):
    """The same clip through the oracles: recurrence in float64, MLP, renderer and their backward
    passes on the CPU, the frames' latent gradients back through time. Bars as for the parts: image
    1e-4, every gradient group max|gpu - oracle| <= 1e-3 max|oracle|."""
    import torch
    import gaussian_splatting_tile_amd as gs
    import synth
    say("[example gradient]")
    cams = [synth.look_at_camera((0.3 * t - 0.3, 0.1, -4.0), (0.0, 0.0, 0.0), 64, 64, 70.0, 70.0) for t in range(3)]
    data = synth.random_scene(500, 7, cams[0], sh_degree=None, scale_lo=0.05, scale_hi=0.2)
    scene = gs.Scene.from_numpy(data)
    target = [i.clone() for i in example.ClipModel(scene, cams, seed=1).render()[0]]
    model = example.ClipModel(scene, cams, seed=2)
    loss = float(model.loss_and_grads(target))
    images = [to_np(i) for i in model.render()[0]]
    torch.cuda.synchronize()

    n, L, H, T = data["n"], model.L, model.H, len(cams)
    x, gate, h0, w = (to_np(p) for p in model.params)
    states = tr.recurrence(gate, x, h0, True)["h"][0]
    scale = 1.0 / sum(t.numel() for t in target)
    d_latents, d_w, want = np.zeros((1, T, L * n)), 0.0, 0.0
    for t, cam in enumerate(cams):
        latent = states[0, t].reshape(L, n).astype(np.float32)
        s = dict(data, rgb=app.forward(cam, data["means"], latent, w, L, H)[0].astype(np.float32))
        f = orc.render_fwd(cam, s)
        assert np.abs(f["image"] - images[t]).max() <= 1e-4
        diff = f["image"] - to_np(target[t])
        want += float((diff.astype(np.float64) ** 2).sum()) * scale
        b = orc.composite_bwd(cam, n, f["ranges"], f["point_list"], f["xy_depth"], f["conic_op"], f["rgb"], f["final_T"],
                              f["n_contrib"], (diff * (2.0 * scale)).astype(np.float32))
        p = orc.preprocess_bwd(cam, s, b["grad_mean2d"], b["grad_conic_op"], b["grad_rgb"])
        g_lat, g_w = app.backward(cam, data["means"], latent, w, L, H, p["grad_rgb_in"])
        d_latents[0, t], d_w = g_lat.reshape(-1), d_w + g_w
    ref = tr.recurrence(gate, x, h0, True, grad_h=d_latents)
    assert abs(loss - want) <= 1e-3 * want
    for name, got, o in (("x", model.grads[0], ref["grad_x"][0]), ("gate", model.grads[1], ref["grad_gate"][0]),
                         ("h0", model.grads[2], ref["grad_h0"][0]), ("weights", model.grads[3], d_w)):
        err, most = np.abs(to_np(got) - o).max(), np.abs(o).max()
        say(f"[example gradient] {name}: {err:.2e} of {most:.2e}")
        assert err <= GRAD_REL * most, (name, err, most)


def test_clip_fit_gets_better(example):
    say("[example fit]")
    losses = example.fit(gaussians=1000, frames=4, steps=30, size=64)
    say(f"[example fit] {losses[0]:.5f} -> {losses[-1]:.5f}")
    assert np.isfinite(losses).all() and losses[-1] < 0.5 * losses[0]
