"""Fits the appearance of a static set of Gaussians to a clip whose colours change with time.

    python examples/fit_clip.py [--gaussians N] [--frames T] [--steps K]

Every Gaussian has a latent that lives through the frames: a gated linear recurrence
(recurrence_fwd) turns per-frame inputs into latents, the appearance MLP turns a frame's latents
into colours, and the rasterizer renders them. The gradient of the squared error goes back the
same way (Rasterizer.backward, appearance_bwd, recurrence_bwd through time), and one Adam step
updates inputs, gates, initial state and MLP weights, with the gradient clipped by its global
norm. The clip to fit is rendered from a hidden model of the same kind.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gaussian_splatting_tile_amd as gs  # noqa: E402
import synth  # noqa: E402


class ClipModel:
    """Latents through time and the MLP that colours them; gradients live in `grads`, in the order of `params`."""

    def __init__(self, scene, cams, n_latent=8, n_hidden=32, seed=0):
        self.scene, self.cams, self.L, self.H = scene, cams, n_latent, n_hidden
        self.T, self.n = len(cams), scene.n
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        f = lambda scale, *d: torch.randn(d, generator=g, device="cuda") * scale
        width = n_latent * self.n  # a frame's [L][n] latents are one step's channels
        self.x, self.gate = f(0.5, 1, self.T, width), f(0.5, 1, self.T, width)
        self.h0 = f(0.5, 1, width)
        self.weights = f(0.3, gs.appearance_params(n_latent, n_hidden))
        self.params = [self.x, self.gate, self.h0, self.weights]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.raster = gs.Rasterizer(capacity=1 << 18)

    def render(self, each=None):
        """The clip's images; with `each`, calls each(t, image, forward state) for every frame."""
        states = gs.recurrence_fwd(self.gate, self.x, h0=self.h0, gating=gs.GATE_SIGMOID, checkpoints=True)
        images = []
        for t, cam in enumerate(self.cams):
            latent = states["h"][0, t].view(self.L, self.n)
            self.scene.rgb = gs.appearance_fwd(cam, self.scene.means, latent, self.weights, self.H)
            out = self.raster.forward(cam, self.scene)
            images.append(out["image"])
            if each is not None:
                each(t, latent, out)
        return images, states

    def loss_and_grads(self, target):
        """Mean squared error against the target clip; fills `grads`."""
        d_latents = torch.empty_like(self.x)
        g_weights = self.grads[3].zero_()
        scale = 1.0 / sum(t.numel() for t in target)
        loss = torch.zeros((), device="cuda")

        def back(t, latent, out):
            diff = out["image"] - target[t]
            loss.add_(diff.square().sum() * scale)
            g = self.raster.backward(self.cams[t], self.scene, out, diff * (2.0 * scale), to_parameters=True)
            a = gs.appearance_bwd(self.cams[t], self.scene.means, latent, self.weights, self.H, g["grad_rgb_in"])
            d_latents[0, t] = a["grad_latent"].view(-1)
            g_weights.add_(a["grad_weights"])

        _, states = self.render(back)
        gs.recurrence_bwd(self.gate, self.x, d_latents, h0=self.h0, ckpt=states["ckpt"], gating=gs.GATE_SIGMOID,
                          out=dict(grad_gate=self.grads[1], grad_x=self.grads[0], grad_h0=self.grads[2]))
        return loss


def fit(gaussians=2000, frames=6, steps=40, size=96, lr=0.03, max_norm=0.01, report=None):
    """Returns the losses of every step. max_norm clips the first, large gradients."""
    cams = [synth.look_at_camera((0.3 * t - 0.6, 0.1, -4.0), (0.0, 0.0, 0.0), size, size, 1.1 * size, 1.1 * size)
            for t in range(frames)]
    data = synth.random_scene(gaussians, 7, cams[0], sh_degree=None, scale_lo=0.02, scale_hi=0.2, spread=1.0)
    scene = gs.Scene.from_numpy(data)
    target = [i.clone() for i in ClipModel(scene, cams, seed=1).render()[0]]
    model = ClipModel(scene, cams, seed=2)
    adam = gs.Adam(model.params, model.grads, lr=[lr, lr, lr, 0.3 * lr], max_norm=max_norm, skip_nonfinite=True)
    losses = []
    for k in range(steps):
        loss = model.loss_and_grads(target)
        norm = adam.step()
        losses.append(float(loss))
        if report is not None:
            report(k, losses[-1], float(norm))
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--gaussians", type=int, default=20000)
    ap.add_argument("--frames", type=int, default=12)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--size", type=int, default=256)
    a = ap.parse_args()
    fit(a.gaussians, a.frames, a.steps, a.size,
        report=lambda k, loss, norm: k % 10 == 0 and print(f"step {k:4d}  loss {loss:.6f}  gradient norm {norm:.2e}",
                                                           flush=True))


if __name__ == "__main__":
    main()
