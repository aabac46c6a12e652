"""Cases of the framework's sequence and training operators: the gated linear recurrence (forward, one step,
forward + backward), the clipping of gradients by their global norm, and the Adam update with that clipping.

Where `own` is false `run` computes them in plain torch operations in 32 bits; where it is true it makes the calls
a user of the package makes. `exact` gives the same outputs in 64 bits, step by step from the definitions.
"""
import math

import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_BETA1, _BETA2, _EPS = 0.9, 0.999, 1e-8


# ---------------------------------------------------------------- cases

def _rec(name, mode, batch, steps, channels, dtype, gating, ragged=False, restarts=False, packed=False):
    c = dict(op="recurrence", mode=mode, batch=batch, steps=steps, channels=channels, dtype=dtype, gating=gating,
             ragged=ragged, restarts=restarts, packed=packed)
    return dict(c, name=name) if name else c


def _opt(name, op, tensors, dtype, max_norm, pdtype="f32", **sizes):
    c = dict(op=op, tensors=tensors, dtype=dtype, max_norm=max_norm, **sizes)
    if op == "adam":
        c["pdtype"] = pdtype
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token for each of 64 running sequences: latency
        _rec("step 64x2048 bf16", "step", 64, 1, 2048, "bf16", "sigmoid"),
        # 8 latents of 160,000 Gaussians through a clip of 16 frames
        _rec("frames 16x1280000 f32", "fwd", 1, 16, 1280000, "f32", "sigmoid"),
        # one long packed sequence of documents, few channels
        _rec("long 65536x1024 bf16", "fwd", 1, 65536, 1024, "bf16", "linear", restarts=True),
        # a training batch with padding; gate and input are halves of one projection
        _rec("train 8x2048x2048 bf16", "train", 8, 2048, 2048, "bf16", "sigmoid", ragged=True, packed=True),
        # odd sizes in float32
        _rec("train 3x1001x777 f32", "train", 3, 1001, 777, "f32", "linear"),
        # the appearance MLP's four tensors (29 latents, 64 hidden units): latency
        _opt("clip mlp f32", "clip", "mlp", "f32", 1.0, latent=29, hidden=64),
        # the parameters of 160,000 Gaussians, SH degree 3
        _opt("clip 160k f32", "clip", "gaussians", "f32", 1.0, n=160000),
        # many tensors of very different sizes, 16-bit gradients
        _opt("clip 300 bf16", "clip", "many", "bf16", 1.0, count=300, largest=1 << 20),
        _opt("adam mlp f32", "adam", "mlp", "f32", 1.0, latent=8, hidden=32),
        # 1,000,000 Gaussians, SH degree 3
        _opt("adam 1M f32", "adam", "gaussians", "f32", 1.0, n=1000000),
        # float32 parameters, 16-bit gradients, many tensors
        _opt("adam 120 bf16 grads", "adam", "many", "bf16", 1.0, count=120, largest=1 << 20),
        # everything in 16 bits but the moments, no clipping
        _opt("adam 40 bf16", "adam", "many", "bf16", 0.0, pdtype="bf16", count=40, largest=1 << 21),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["step", "fwd", "train", "clip", "adam"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if kind == "step":
        return _rec(None, "step", _log(rng, 1, 256), 1, _log(rng, 64, 8192), dtype, rng.choice(["linear", "sigmoid"]))
    if kind in ("fwd", "train"):
        steps = _log(rng, 2, 65536)
        room = (1 << 26) if kind == "fwd" else (1 << 25)
        channels = _log(rng, 64, max(64, min(1 << 20, room // steps)))
        batch = _log(rng, 1, max(1, min(16, room // (steps * channels))))
        return _rec(None, kind, batch, steps, channels, dtype, rng.choice(["linear", "sigmoid"]), rng.random() < 0.5,
                    rng.random() < 0.5, rng.random() < 0.5)
    max_norm = rng.choice([0.5, 1.0, 1e9])
    sets = rng.choice(["mlp", "gaussians", "many"])
    pdtype = rng.choice(["f32", dtype])
    if sets == "mlp":
        return _opt(None, kind, sets, dtype, max_norm, pdtype, latent=rng.randint(1, 29), hidden=rng.randint(1, 64))
    if sets == "gaussians":
        return _opt(None, kind, sets, dtype, max_norm, pdtype, n=_log(rng, 1000, 1000000))
    return _opt(None, kind, sets, dtype, max_norm, pdtype, count=_log(rng, 2, 300), largest=_log(rng, 1 << 8, 1 << 20))


# ---------------------------------------------------------------- inputs

def _sizes(case):
    """Element counts of a case's tensors; of the sizes of "many" the k-th is largest * 2^-(10 k / count), made odd."""
    if case["tensors"] == "mlp":
        latent, hidden = case["latent"], case["hidden"]
        return [hidden * (latent + 3), hidden, 3 * hidden, 3]
    if case["tensors"] == "gaussians":
        n = case["n"]
        return [3 * n, 3 * n, 4 * n, n, 48 * n]  # means, scales, quats, opacity, SH
    count, largest = case["count"], case["largest"]
    return [max(1, int(largest * 2.0 ** (-10.0 * ((7 * k) % count) / count))) | 1 for k in range(count)]


def _split(flat, sizes):
    return list(torch.split(flat, sizes))


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "recurrence":
        B, T, D, t = case["batch"], case["steps"], case["channels"], _TYPES[case["dtype"]]
        f = lambda *d: torch.randn(d, generator=g, device=_DEV)  # noqa: E731
        # forgetting gates: most remember for tens of steps, some for thousands
        z, x = f(B, T, D).mul_(1.5).add_(3.0), f(B, T, D)
        if case["gating"] == "linear":
            z.sigmoid_()
        if case["packed"]:
            both = torch.cat([z, x], 2).to(t)
            s["gate"], s["x"] = both[:, :, :D], both[:, :, D:]
        else:
            s["gate"], s["x"] = z.to(t), x.to(t)
        del z, x
        s["h0"] = f(B, D)
        s["lengths"] = s["restart"] = None
        if case["ragged"]:
            lengths = torch.randint(0, T + 1, (B,), generator=g, device=_DEV, dtype=torch.int32)
            lengths[0] = T
            if B > 2:
                lengths[1], lengths[2] = 0, 1
            s["lengths"] = lengths
        if case["restarts"]:
            s["restart"] = (torch.rand((B, T), generator=g, device=_DEV) < 16.0 / (T + 16)).to(torch.uint8)
        if case["mode"] == "train":
            s["grad_h"], s["grad_last"] = f(B, T, D).to(t), f(B, D)
        return s
    sizes, t = _sizes(case), _TYPES[case["dtype"]]
    N = sum(sizes)
    f = lambda: torch.randn(N, generator=g, device=_DEV)  # noqa: E731
    # gradients whose scale differs from tensor to tensor, above the clipping norm together
    scale = torch.rand(len(sizes), generator=g, device=_DEV).mul_(4.0).exp_().mul_(0.01)
    grad = f() * torch.repeat_interleave(scale, torch.tensor(sizes, device=_DEV), output_size=N)
    s["flat_grad"] = grad.to(t)
    s["grads"] = _split(s["flat_grad"], sizes)
    if case["op"] == "clip":
        s["flat_out"] = torch.empty_like(s["flat_grad"])
        s["outs"] = _split(s["flat_out"], sizes)
        if own:
            import gaussian_splatting_tile_amd as gs
            s["list"] = gs.GradList(s["grads"], out=s["outs"])
        return s
    s["flat_param"] = f().to(_TYPES[case["pdtype"]])
    s["flat_m"] = grad * 0.1
    s["flat_v"] = grad.square().mul_(0.01).add_(1e-6)
    s["params"], s["m"], s["v"] = (_split(s[k], sizes) for k in ("flat_param", "flat_m", "flat_v"))
    # a rate and a decay for each tensor, as parameters of different kinds have them
    s["lr"] = [1e-3 * (1 + k % 5) for k in range(len(sizes))]
    s["weight_decay"] = [0.01 * (k % 2) for k in range(len(sizes))]
    s["taken"] = 100
    if own:
        import gaussian_splatting_tile_amd as gs
        s["adam"] = gs.Adam(s["params"], s["grads"], lr=s["lr"], betas=(_BETA1, _BETA2), eps=_EPS,
                            weight_decay=s["weight_decay"], max_norm=case["max_norm"], exp_avg=s["m"],
                            exp_avg_sq=s["v"], step=s["taken"])
    return s


# ---------------------------------------------------------------- one pass

def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, by recursive doubling."""
    d = 1
    while d < a.shape[1]:
        nb = b.clone()
        nb[:, d:].addcmul_(a[:, d:], b[:, :-d])
        if 2 * d < a.shape[1]:
            na = a.clone()
            na[:, d:].mul_(a[:, :-d])
            a = na
        b, d = nb, 2 * d
    return b


def _plain_recurrence(s):
    case, t = s["case"], _TYPES[s["case"]["dtype"]]
    gate, x, h0 = s["gate"].float(), s["x"].float(), s["h0"]
    B, T, D = gate.shape
    sigmoid = case["gating"] == "sigmoid"
    a = torch.sigmoid(gate) if sigmoid else gate
    rest = torch.sigmoid(-gate) if sigmoid else None  # 1 - a without cancellation
    u = rest * x if sigmoid else x
    ae = a
    if s["restart"] is not None:
        ae = torch.where(s["restart"].bool()[:, :, None], 0.0, ae)
    valid = last = None
    if s["lengths"] is not None:
        valid = (torch.arange(T, device=gate.device)[None, :] < s["lengths"][:, None])[:, :, None]
        last = (s["lengths"].long() - 1).clamp_min(0)[:, None, None].expand(B, 1, D)
        ae, u = torch.where(valid, ae, 0.0), torch.where(valid, u, 0.0)
        some = (s["lengths"] > 0)[:, None]
    first = u[:, :1] + ae[:, :1] * h0[:, None]
    h = _doubling(ae, torch.cat([first, u[:, 1:]], 1))
    h_last = h[:, -1].clone() if valid is None else torch.where(some, h.gather(1, last)[:, 0], h0)
    if case["mode"] != "train":
        return dict(h=h.to(t), h_last=h_last)
    g = s["grad_h"].float()
    if valid is None:
        g = torch.cat([g[:, :-1], (g[:, -1] + s["grad_last"])[:, None]], 1)
    else:
        g = torch.where(valid, g, 0.0).scatter_add(1, last, torch.where(some, s["grad_last"], 0.0)[:, None])
    # d_t = g_t + a_{t+1} d_{t+1}: the same recurrence from the other end
    nxt = torch.cat([ae[:, 1:], torch.zeros_like(ae[:, :1])], 1)
    d = _doubling(nxt.flip(1), g.flip(1)).flip(1)
    grad_h0 = ae[:, 0] * d[:, 0]
    if valid is not None:
        grad_h0 = torch.where(some, grad_h0, s["grad_last"])
    prev = torch.cat([h0[:, None], h[:, :-1]], 1)
    if s["restart"] is not None:
        prev = torch.where(s["restart"].bool()[:, :, None], 0.0, prev)
    dg = d * (prev - x) * (a * rest) if sigmoid else d * prev
    dx = d * rest if sigmoid else d
    if valid is not None:
        dg, dx = torch.where(valid, dg, 0.0), torch.where(valid, dx, 0.0)
    return dict(h=h.to(t), h_last=h_last, grad_gate=dg.to(t), grad_x=dx.to(t), grad_h0=grad_h0)


def _plain_norm(s):
    return s["flat_grad"].float().square().sum().sqrt()


def _plain_clip(s):
    norm = _plain_norm(s)
    coef = (s["case"]["max_norm"] / (norm + 1e-6)).clamp_max(1.0)
    s["flat_out"].copy_(s["flat_grad"].float() * coef)
    return dict(out=s["flat_out"], norm=norm)


def _plain_adam(s):
    case = s["case"]
    s["taken"] += 1
    out = dict(param=s["flat_param"], m=s["flat_m"], v=s["flat_v"])
    grad = s["flat_grad"].float()
    if case["max_norm"] > 0:
        out["norm"] = _plain_norm(s)
        grad = grad * (case["max_norm"] / (out["norm"] + 1e-6)).clamp_max(1.0)
    s["flat_m"].mul_(_BETA1).add_(grad, alpha=1 - _BETA1)
    s["flat_v"].mul_(_BETA2).addcmul_(grad, grad, value=1 - _BETA2)
    bc1, bc2 = 1 - _BETA1 ** s["taken"], 1 - _BETA2 ** s["taken"]
    step = (s["flat_m"] / bc1) / ((s["flat_v"] / bc2).sqrt() + _EPS)
    for p, d, lr, wd in zip(s["params"], _split(step, [p.numel() for p in s["params"]]), s["lr"], s["weight_decay"]):
        p.copy_(p.float() * (1 - lr * wd) - lr * d)
    return out


def _own_recurrence(s):
    import gaussian_splatting_tile_amd as gs
    mode = s["case"]["mode"]
    gating = gs.GATE_SIGMOID if s["case"]["gating"] == "sigmoid" else gs.GATE_LINEAR
    if mode == "step":
        out = gs.recurrence_fwd(s["gate"], s["x"], h0=s["h0"], gating=gating)
        return dict(h=out["h"], h_last=out["h_last"])
    shape = dict(gating=gating, lengths=s["lengths"], restart=s["restart"])
    out = gs.recurrence_fwd(s["gate"], s["x"], h0=s["h0"], checkpoints=mode == "train", **shape)
    if mode == "fwd":
        return dict(h=out["h"], h_last=out["h_last"])
    back = gs.recurrence_bwd(s["gate"], s["x"], s["grad_h"], h0=s["h0"], ckpt=out["ckpt"], grad_last=s["grad_last"],
                             **shape)
    return dict(h=out["h"], h_last=out["h_last"], grad_gate=back["grad_gate"], grad_x=back["grad_x"],
                grad_h0=back["grad_h0"])


def run(state):
    op = state["case"]["op"]
    if not own:
        return (_plain_recurrence if op == "recurrence" else _plain_clip if op == "clip" else _plain_adam)(state)
    if op == "recurrence":
        return _own_recurrence(state)
    if op == "clip":
        return dict(out=state["flat_out"], norm=state["list"].clip(state["case"]["max_norm"]))
    norm = state["adam"].step()
    out = dict(param=state["flat_param"], m=state["flat_m"], v=state["flat_v"])
    if state["case"]["max_norm"] > 0:
        out["norm"] = norm
    return out


# ---------------------------------------------------------------- work and exact values

def work(case):
    if case["op"] == "recurrence":
        E, s = case["batch"] * case["steps"] * case["channels"], _BYTES[case["dtype"]]
        state = 4 * case["batch"] * case["channels"]
        read = 0.5 if case["ragged"] else 1.0  # the mean share of the steps that the lengths leave
        ops = 2 + (4 if case["gating"] == "sigmoid" else 0)
        if case["mode"] == "train":
            return {"bytes": (3 + 3 * read) * E * s + 4 * state, "flops": (2 * ops + 4) * E * read}
        return {"bytes": (1 + 2 * read) * E * s + 2 * state, "flops": ops * E * read}
    N, s = sum(_sizes(case)), _BYTES[case["dtype"]]
    if case["op"] == "clip":
        return {"bytes": 2 * N * s, "flops": 3 * N}
    return {"bytes": N * (16 + s + 2 * _BYTES[case["pdtype"]]), "flops": 16 * N}


def _exact_recurrence(s):
    case = s["case"]
    z, x, h = s["gate"].double(), s["x"].double(), s["h0"].double()
    B, T, D = z.shape
    a = z if case["gating"] == "linear" else 1 / (1 + torch.exp(-z))
    u = x if case["gating"] == "linear" else x / (1 + torch.exp(z))
    keep = torch.ones((B, T, 1), dtype=torch.bool, device=z.device)  # steps that carry the state on
    if s["restart"] is not None:
        keep &= s["restart"][:, :, None] == 0
    n = s["lengths"] if s["lengths"] is not None else torch.full((B,), T, device=z.device)
    live = torch.arange(T, device=z.device)[None, :, None] < n[:, None, None]
    hs, prev = torch.zeros_like(z), torch.zeros_like(z)
    for t in range(T):
        prev[:, t] = torch.where(keep[:, t], h, 0.0)
        h = torch.where(live[:, t], a[:, t] * prev[:, t] + u[:, t], h)
        hs[:, t] = torch.where(live[:, t], h, 0.0)
    out = dict(h=hs, h_last=h)
    if case["mode"] != "train":
        return out
    g, d = s["grad_h"].double(), s["grad_last"].double()
    dz, dx = torch.zeros_like(z), torch.zeros_like(z)
    for t in range(T - 1, -1, -1):
        here = d + g[:, t]
        if case["gating"] == "linear":
            dz[:, t], dx[:, t] = here * prev[:, t], here
        else:
            rest = 1 / (1 + torch.exp(z[:, t]))
            dz[:, t], dx[:, t] = here * (prev[:, t] - x[:, t]) * a[:, t] * rest, here * rest
        d = torch.where(live[:, t], torch.where(keep[:, t], a[:, t] * here, 0.0), d)
    return dict(out, grad_gate=torch.where(live, dz, 0.0), grad_x=torch.where(live, dx, 0.0), grad_h0=d)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "recurrence":
        return _exact_recurrence(s)
    g = s["flat_grad"].double()
    norm = torch.linalg.vector_norm(g)
    coef = min(1.0, case["max_norm"] / (float(norm) + 1e-6)) if case["op"] == "clip" or case["max_norm"] > 0 else 1.0
    if case["op"] == "clip":
        return dict(out=g * coef, norm=norm)
    g = g * coef
    m = _BETA1 * s["flat_m"].double() + (1 - _BETA1) * g
    v = _BETA2 * s["flat_v"].double() + (1 - _BETA2) * g ** 2
    t = s["taken"] + 1
    by = lambda values: torch.repeat_interleave(torch.tensor(values, dtype=torch.float64, device=g.device),  # noqa: E731
                                                torch.tensor(_sizes(case), device=g.device))
    lr, wd = by(s["lr"]), by(s["weight_decay"])
    p = s["flat_param"].double()
    p = p - lr * wd * p - lr * (m / (1 - _BETA1 ** t)) / (torch.sqrt(v / (1 - _BETA2 ** t)) + _EPS)
    out = dict(param=p, m=m, v=v)
    return dict(out, norm=norm) if case["max_norm"] > 0 else out
