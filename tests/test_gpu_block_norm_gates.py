"""Gates of the block norms far from 0, element by element.

Tolerance. u = 2^-24 is float32's unit roundoff; the hardware's exponential and reciprocal are off by an ulp, 2 u. With q =
exp(-|z|) (the exponential 2 u, the correction of its argument u), 1 + q (u more), its reciprocal (2 u) and the product
(u), q / (1 + q) is off by at most 3 + 2.5 + 2 + 1 = 8.5 u, and 1 less that, which is at least 1/2, by 9.5 u. The
slope's product of the two is off by 12 u, and up to 4 products follow: 16 u of each term. 16-bit types: the exponential's
argument rounded, |z| u (log2(e) and the product, half of it each), and the rounding at the end; what is under float32's
smallest normal number, or half of the type's smallest subnormal, may be 0."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# unit roundoff of the type, and what may be lost in any case
TYPES = dict(f32=(0.0, 2.0 ** -126), bf16=(2.0 ** -8, 2.0 ** -126), f16=(2.0 ** -11, 2.0 ** -25))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [3, 512, 777, 8192])
@pytest.mark.parametrize("gating", ["sigmoid", "silu"])
def test_gates_far_from_zero(gating, width, dtype):
    import torch
    import gaussian_splatting_tile_amd as gs
    rng = np.random.default_rng(width)
    z = 87 * rng.uniform(-1, 1, (40, width)) * 10.0 ** -rng.uniform(0, 3, (40, width))
    y, up = (rng.uniform(1, 2, z.shape) for _ in range(2))
    t, (u, tiny) = dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[dtype], TYPES[dtype]
    g = dict(gating=gs.BLOCK_GATE_SILU if gating == "silu" else gs.BLOCK_GATE_SIGMOID)
    dev = [torch.tensor(x, device="cuda").to(t) for x in (y, up, z)]
    out = gs.block_norm_fwd(dev[0], gate=dev[2], **g)["out"].double().cpu().numpy()
    back = gs.block_norm_bwd(dev[0], dev[1], gate=dev[2], **g)
    y, up, z = (x.double().cpu().numpy() for x in dev)
    tol = 16 * U + (0 if dtype == "f32" else u + np.abs(z) * U)
    sg, other = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    act, terms = (z * sg, (sg, z * sg * other)) if gating == "silu" else (sg, (sg * other,))
    assert (np.abs(out - act * y) <= tol * np.abs(act * y) + tiny).all()
    assert (np.abs(back["grad_y"].double().cpu().numpy() - act * up) <= tol * np.abs(act * up) + tiny).all()
    far = np.abs(back["grad_gate"].double().cpu().numpy() - sum(terms) * y * up)
    assert (far <= tol * sum(np.abs(t) for t in terms) * y * up + tiny).all()


@pytest.mark.parametrize("gating", ["sigmoid", "silu"])
def test_gates_that_are_not_finite(gating):
    """As the formulas have it: sigmoid is 0 and 1 at the infinities, and a NaN stays one."""
    import torch
    import gaussian_splatting_tile_amd as gs
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[-inf, -1e30, -200.0, 0.0, 200.0, 1e30, inf, nan]], device="cuda")
    kind = gs.BLOCK_GATE_SILU if gating == "silu" else gs.BLOCK_GATE_SIGMOID
    out = gs.block_norm_fwd(torch.ones_like(z), gate=z, gating=kind)["out"][0].cpu()
    want = [0.0, 0.0, 0.0, 0.5, 1.0, 1.0, 1.0, nan] if gating == "sigmoid" else [nan, 0.0, 0.0, 0.0, 200.0, 1e30, inf, nan]
    assert torch.equal(out.nan_to_num(7.0, inf, -inf), torch.tensor(want).nan_to_num(7.0, inf, -inf))
