"""Cases of the framework's gated delta rule (forward, few new tokens, forward + backward) and of the norms around a
block: the block's output normalised, gated, scaled and added to the residual stream, and the next block's norm of
that sum (forward, forward + backward).

Where `own` is false `run` computes them in plain torch operations in 32 bits (the delta rule in chunks of 64 steps,
with its decays' sums in 64; a few new tokens step by step); where it is true it makes the calls a user of the package
makes. `exact` gives the same outputs in 64 bits: the delta rule step by step from its definition, the norms by
differentiating theirs.
"""
import math

import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_EPS = 1e-5
_CHUNK = 64


# ---------------------------------------------------------------- cases

def _delta(name, mode, batch, steps, key_heads, heads, dk, dv, dtype, ragged=False, restarts=False, packed=False):
    c = dict(op="delta", mode=mode, batch=batch, steps=steps, key_heads=key_heads, heads=heads, dk=dk, dv=dv,
             dtype=dtype, ragged=ragged, restarts=restarts, packed=packed)
    return dict(c, name=name) if name else c


def _norm(name, mode, rows, width, dtype, post, gating, residual, scale, pre, heads=1, packed=False):
    c = dict(op="norm", mode=mode, rows=rows, width=width, dtype=dtype, post=post, gating=gating, residual=residual,
             scale=scale, pre=pre, heads=heads, packed=packed)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of one sequence, small heads: latency
        _delta("delta step 1x8 64x64 f32", "step", 1, 1, 4, 8, 64, 64, "f32"),
        # one new token for each of 64 running sequences: their states are read and written
        _delta("delta step 64x16 128x128 bf16", "step", 64, 1, 8, 16, 128, 128, "bf16", packed=True),
        # one prompt, two value heads for each key head
        _delta("delta prompt 8192 16/32x128 bf16", "fwd", 1, 8192, 16, 32, 128, 128, "bf16", packed=True),
        # one long packed sequence of documents, few heads
        _delta("delta long 65536 4x128 f16", "fwd", 1, 65536, 4, 4, 128, 128, "f16", restarts=True),
        # a training batch with padding; q, k and v are parts of one projection
        _delta("delta train 8x2048 8/16x128 bf16", "train", 8, 2048, 8, 16, 128, 128, "bf16", ragged=True, packed=True),
        # odd sizes in float32
        _delta("delta train 3x777 5x96x80 f32", "train", 3, 777, 5, 5, 96, 80, "f32", restarts=True),
        # one new token for each of 64 running sequences: latency
        _norm("norm 64x2048 bf16", "fwd", 64, 2048, "bf16", "rms", "none", True, False, "rms"),
        # a prompt's tokens, a wide stream
        _norm("norm 8192x8192 f16", "fwd", 8192, 8192, "f16", "rms", "sigmoid", True, True, "rms"),
        # a training step's tokens, everything in use
        _norm("norm train 16384x2048 bf16", "train", 16384, 2048, "bf16", "rms", "sigmoid", True, True, "rms"),
        # the heads' outputs of a recurrent block, gated by a part of a projection
        _norm("norm train 16384x16 heads x128 bf16", "train", 16384, 128, "bf16", "rms", "silu", False, False, "none",
              heads=16, packed=True),
        # odd sizes in float32, means taken out
        _norm("norm train 1001x777 f32", "train", 1001, 777, "f32", "layer", "none", True, True, "layer"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["f32", "bf16", "f16"])
    if rng.random() < 0.55:
        mode = rng.choice(["step", "fwd", "train"])
        dk, dv = rng.choice([rng.randint(16, 128), 64, 128]), rng.choice([rng.randint(16, 128), 64, 128])
        key_heads, group = _log(rng, 1, 16), rng.choice([1, 1, 2, 3])
        if mode == "step":
            return _delta(None, mode, _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 5]), key_heads, key_heads * group, dk,
                          dv, dtype, packed=rng.random() < 0.5)
        steps = _log(rng, 2, 32768 if mode == "fwd" else 8192)
        room = (1 << 18) if mode == "fwd" else (1 << 17)
        heads = max(1, min(key_heads, room // (steps * group)))
        batch = _log(rng, 1, max(1, min(8, room // (steps * heads * group))))
        return _delta(None, mode, batch, steps, heads, heads * group, dk, dv, dtype, rng.random() < 0.5,
                      rng.random() < 0.5, rng.random() < 0.5)
    mode = rng.choice(["fwd", "train"])
    if rng.random() < 0.35:
        heads, width = rng.choice([1, 4, 8, 16, 32]), rng.choice([rng.randint(16, 256), 64, 128])
        rows = _log(rng, 1, (1 << 24) // (heads * width))
        return _norm(None, mode, rows, width, dtype, rng.choice(["rms", "layer"]), rng.choice(["none", "sigmoid", "silu"]),
                     False, False, "none", heads, rng.random() < 0.5)
    width = _log(rng, 64, 16384)
    rows = _log(rng, 1, min(32768, (1 << 25) // width))
    return _norm(None, mode, rows, width, dtype, rng.choice(["none", "rms", "layer"]),
                 rng.choice(["none", "sigmoid", "silu"]), True, rng.random() < 0.5, rng.choice(["rms", "layer"]), 1,
                 rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    f = lambda *d: torch.randn(d, generator=g, device=_DEV)  # noqa: E731
    t, s = _TYPES[case["dtype"]], dict(case=case)
    if case["op"] == "delta":
        B, T, Hk, H, dk, dv = (case[k] for k in ("batch", "steps", "key_heads", "heads", "dk", "dv"))
        unit = lambda z: z.div_(z.square().sum(-1, keepdim=True).add_(1e-6).sqrt_())  # noqa: E731
        act = lambda z: z * torch.sigmoid(z)  # noqa: E731
        # queries and keys are unit vectors behind an activation that leaves their mean above 0
        q, k, v = unit(act(f(B, T, Hk, dk))), unit(act(f(B, T, Hk, dk))), act(f(B, T, H, dv))
        if case["packed"]:
            rows = torch.cat([q.view(B, T, -1), k.view(B, T, -1), v.view(B, T, -1)], 2).to(t)
            q, k, v = rows.split([Hk * dk, Hk * dk, H * dv], 2)
            s.update(q=q.unflatten(2, (Hk, dk)), k=k.unflatten(2, (Hk, dk)), v=v.unflatten(2, (H, dv)))
        else:
            s.update(q=q.to(t), k=k.to(t), v=v.to(t))
        del q, k, v
        # most heads forget over tens of steps, some over thousands
        s["log_decay"] = f(B, T, H).mul_(0.7).add_(f(H).mul_(1.5)).sub_(3.5).exp_().neg_()
        s["beta"] = torch.sigmoid(f(B, T, H))
        s["h0"] = f(B, H, dk, dv).mul_(0.2)
        s["scale"] = dk ** -0.5
        s["lengths"] = s["restart"] = None
        if case["ragged"]:
            lengths = torch.randint(0, T + 1, (B,), generator=g, device=_DEV, dtype=torch.int32)
            lengths[0] = T
            if B > 2:
                lengths[1], lengths[2] = 0, 1
            s["lengths"] = lengths
        if case["restarts"]:
            s["restart"] = (torch.rand((B, T), generator=g, device=_DEV) < 8.0 / (T + 8)).to(torch.uint8)
        if case["mode"] == "train":
            s["grad_o"], s["grad_last"] = f(B, T, H, dv).to(t), f(B, H, dk, dv).mul_(0.1)
        return s
    R, D, H = case["rows"], case["width"], case["heads"]
    shape = (R, H, D) if H > 1 else (R, D)
    y, z = f(*shape).mul_(1.0 + f(R, *([1] * (len(shape) - 1))).abs_()), f(*shape)
    if case["packed"]:
        both = torch.cat([y.view(R, -1), z.view(R, -1)], 1).to(t)
        s["y"], s["gate"] = both[:, :H * D].view(R, *shape[1:]), both[:, H * D:].view(R, *shape[1:])
    else:
        s["y"], s["gate"] = y.to(t), z.to(t)
    if case["gating"] == "none":
        s["gate"] = None
    s["residual"] = f(*shape).mul_(3.0).to(t) if case["residual"] else None
    weight = lambda: f(D).mul_(0.2).add_(1.0)  # noqa: E731
    s["post_weight"] = weight() if case["post"] != "none" else None
    s["post_bias"] = f(D).mul_(0.1) if case["post"] == "layer" else None
    s["scale"] = weight().mul_(0.3) if case["scale"] else None
    s["pre_weight"] = weight() if case["pre"] != "none" else None
    s["pre_bias"] = f(D).mul_(0.1) if case["pre"] == "layer" else None
    if case["mode"] == "train":
        s["grad_out"] = f(*shape).to(t)
        s["grad_norm"] = f(*shape).to(t) if case["pre"] != "none" else None
    return s


# ---------------------------------------------------------------- the delta rule, plain

def _unit_lower_inverse(a):
    """(I + a)^-1 of strictly lower triangular a [..., 64, 64]: the diagonal blocks' inverses, joined pair by pair."""
    n = a.shape[-1]
    inv = torch.eye(n, device=a.device, dtype=a.dtype).expand_as(a).contiguous()
    w = 1
    while w < n:
        m = n // (2 * w)
        b = a.unflatten(-2, (m, 2, w)).unflatten(-1, (m, 2, w))  # [..., m, 2, w, m, 2, w]
        i = inv.unflatten(-2, (m, 2, w)).unflatten(-1, (m, 2, w))
        d = torch.arange(m, device=a.device)
        low = b[..., d, 1, :, d, 0, :]  # [m, ..., w, w]
        i[..., d, 1, :, d, 0, :] = -(i[..., d, 1, :, d, 1, :] @ (low @ i[..., d, 0, :, d, 0, :]))
        w *= 2
    return inv


def _plain_steps(s):
    """A few steps, one after another."""
    case = s["case"]
    r, S, o = case["heads"] // case["key_heads"], s["h0"], []
    q, k, v = s["q"].float() * s["scale"], s["k"].float(), s["v"].float()
    if r > 1:
        q, k = q.repeat_interleave(r, 2), k.repeat_interleave(r, 2)
    a, beta = s["log_decay"].exp()[..., None, None], s["beta"][..., None]
    for t in range(case["steps"]):
        S = S * a[:, t]
        u = beta[:, t] * (v[:, t] - (S * k[:, t, :, :, None]).sum(-2))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        o.append((S * q[:, t, :, :, None]).sum(-2))
    return dict(o=torch.stack(o, 1).to(_TYPES[case["dtype"]]), h_last=S)


def _plain_delta(s):
    case, C = s["case"], _CHUNK
    if case["mode"] == "step":
        return _plain_steps(s)
    t = _TYPES[case["dtype"]]
    B, T, Hk, H, dk, dv = (case[x] for x in ("batch", "steps", "key_heads", "heads", "dk", "dv"))
    r, n = H // Hk, -(-T // C)
    N, pad = B * H, n * C - T
    dev = s["q"].device
    live = torch.ones((B, T), dtype=torch.bool, device=dev)
    if s["lengths"] is not None:
        live = torch.arange(T, device=dev)[None, :] < s["lengths"][:, None]

    def chunks(x, heads_of=1):
        """[B, T, heads, ...] -> [B H, n, C, ...] in 32 bits, 0 at padding."""
        x = torch.where(live.view(B, T, *[1] * (x.dim() - 2)), x.float(), 0.0)
        x = torch.cat([x, x.new_zeros(B, pad, *x.shape[2:])], 1).transpose(1, 2)
        return x.repeat_interleave(heads_of, 1).reshape(N, n, C, *x.shape[3:])

    def back(x):
        """The inverse, for x [B H, n, C, ...]."""
        return x.reshape(B, H, n * C, *x.shape[3:])[:, :, :T].transpose(1, 2)

    q, k, v = chunks(s["q"], r) * s["scale"], chunks(s["k"], r), chunks(s["v"])
    beta, g = chunks(s["beta"])[..., None], chunks(s["log_decay"])
    cut = torch.zeros((B, n * C), dtype=torch.long, device=dev)
    if s["restart"] is not None:
        cut[:, :T] = (s["restart"].bool() & live).long()
    seg = cut.view(B, 1, n, C).cumsum(-1).expand(B, H, n, C).reshape(N, n, C)
    G = g.double().cumsum(-1)
    # decays in 64 bits up to their exponential: from j to i, from the chunk's start, to its end, over all of it
    same = (seg[..., :, None] == seg[..., None, :]).tril()
    D = torch.where(same, (G[..., :, None] - G[..., None, :]).float(), -torch.inf).exp()
    first = torch.where(seg == 0, G.float().exp(), 0.0)[..., None]
    end = D[..., -1, :, None]
    whole = first[..., -1:, :]
    kt = k.transpose(-1, -2)
    A = (beta * D * (k @ kt)).tril(-1)
    P = D * (q @ kt)
    M = _unit_lower_inverse(A)
    W, U0, ke = M @ (beta * first * k), M @ (beta * v), end * k
    ket = ke.transpose(-1, -2).contiguous()
    S = s["h0"].reshape(N, dk, dv)
    S0, U = k.new_empty(N, n, dk, dv), torch.empty_like(U0)
    for c in range(n):
        S0[:, c] = S
        U[:, c] = U0[:, c] - W[:, c] @ S
        S = whole[:, c] * S + ket[:, c] @ U[:, c]
    o = first * (q @ S0) + P @ U
    out = dict(o=back(o).to(t), h_last=S.view(B, H, dk, dv))
    if case["mode"] != "train":
        return out
    do = chunks(s["grad_o"])
    dS = s["grad_last"].reshape(N, dk, dv)
    Mt = M.transpose(-1, -2)
    dU, dSe, dR = P.transpose(-1, -2) @ do, torch.empty_like(S0), torch.empty_like(U0)
    add = (first * q).transpose(-1, -2) @ do
    bk = (beta * first * k).transpose(-1, -2)
    for c in range(n - 1, -1, -1):
        dSe[:, c] = dS
        dR[:, c] = Mt[:, c] @ (dU[:, c] + ke[:, c] @ dS)
        dS = whole[:, c] * dS + add[:, c] - bk[:, c] @ dR[:, c]
    Ut, S0t = U.transpose(-1, -2), S0.transpose(-1, -2)
    dP, dA = (do @ Ut) * D, -(dR @ Ut).tril(-1)
    qs, ks, us = first * (do @ S0t), beta * first * (dR @ S0t), end * (U @ dSe.transpose(-1, -2))
    X = dP * (q @ kt) + dA * A
    dA = dA * beta * D
    dq = (dP @ k + qs) * s["scale"]
    dk_ = dP.transpose(-1, -2) @ q + dA @ k + dA.transpose(-1, -2) @ k - ks + us
    dbeta = (dR * (v - first * (k @ S0))).sum(-1) + ((-(dR @ Ut)).tril(-1) * D * (k @ kt)).sum(-1)
    # the decay of step t lies between every j < t <= i, between the state in front and every i >= t, and between
    # every j < t and the state behind; the factors of pairs that a restart parts are 0
    fro, aft, all_ = (q * qs - k * ks).sum(-1), (k * us).sum(-1), whole[..., 0, 0] * (S0 * dSe).sum((-1, -2))
    lo = X.new_zeros(X.shape)
    lo[..., 1:] = X.cumsum(-1)[..., :-1]
    early = X.new_zeros(aft.shape)
    early[..., 1:] = aft.cumsum(-1)[..., :-1]
    dg = lo.tril().sum(-2) + fro.flip(-1).cumsum(-1).flip(-1) + early + all_[..., None]
    shared = lambda x: back(x).unflatten(2, (Hk, r)).sum(3)  # noqa: E731
    here = live[:, :, None]
    out.update(grad_q=shared(dq).to(t), grad_k=shared(dk_).to(t), grad_v=back(beta * dR).to(t),
               grad_log_decay=torch.where(here, back(dg), 0.0), grad_beta=torch.where(here, back(dbeta), 0.0),
               grad_h0=dS.view(B, H, dk, dv))
    return out


# ---------------------------------------------------------------- the norms, plain

def _plain_one(x, kind):
    """x normalised over the last dimension, and 1 / its deviation."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = (x.square().mean(-1, keepdim=True) + _EPS).rsqrt()
    return x * r, r


def _plain_one_back(d, xhat, r, kind):
    dx = d - xhat * (d * xhat).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - d.mean(-1, keepdim=True)
    return dx * r


def _plain_norm(s):
    case = s["case"]
    t, post, pre, train = _TYPES[case["dtype"]], case["post"], case["pre"], case["mode"] == "train"
    y = s["y"].float()
    h, act, sig, z = y, None, None, None
    if post != "none":
        yhat, ry = _plain_one(y, post)
        h = yhat * s["post_weight"]
        if post == "layer":
            h = h + s["post_bias"]
    b = h
    if case["gating"] != "none":
        z = s["gate"].float()
        sig = torch.sigmoid(z)
        act = sig if case["gating"] == "sigmoid" else z * sig
        b = h * act
    u = b * s["scale"] if case["scale"] else b
    x = u if s["residual"] is None else s["residual"].float() + u
    out = dict(out=x.to(t))
    if pre != "none":
        xhat, rx = _plain_one(x, pre)
        n = xhat * s["pre_weight"]
        out["norm"] = (n + s["pre_bias"] if pre == "layer" else n).to(t)
    if not train:
        return out
    cols = lambda v: v.reshape(-1, v.shape[-1]).sum(0)  # noqa: E731
    d = s["grad_out"].float()
    if pre != "none":
        dn = s["grad_norm"].float()
        out["grad_pre_weight"] = cols(dn * xhat)
        if pre == "layer":
            out["grad_pre_bias"] = cols(dn)
        d = d + _plain_one_back(dn * s["pre_weight"], xhat, rx, pre)
    if s["residual"] is not None:
        out["grad_residual"] = d.to(t)
    if case["scale"]:
        out["grad_scale"] = cols(d * b)
        d = d * s["scale"]
    if act is not None:
        dz = d * h * sig * (1 - sig) if case["gating"] == "sigmoid" else d * h * sig * (1 + z * (1 - sig))
        out["grad_gate"] = dz.to(t)
        d = d * act
    if post != "none":
        out["grad_post_weight"] = cols(d * yhat)
        if post == "layer":
            out["grad_post_bias"] = cols(d)
        d = _plain_one_back(d * s["post_weight"], yhat, ry, post)
    out["grad_y"] = d.to(t)
    return out


# ---------------------------------------------------------------- one pass

def _own_delta(s):
    import gaussian_splatting_tile_amd as gs
    mode, a = s["case"]["mode"], (s["q"], s["k"], s["v"], s["log_decay"], s["beta"])
    shape = dict(h0=s["h0"], scale=s["scale"], lengths=s["lengths"], restart=s["restart"])
    out = gs.delta_rule_fwd(*a, checkpoints=mode == "train", **shape)
    if mode != "train":
        return dict(o=out["o"], h_last=out["h_last"])
    back = gs.delta_rule_bwd(*a, s["grad_o"], ckpt=out["ckpt"], grad_last=s["grad_last"], **shape)
    return dict(back, o=out["o"], h_last=out["h_last"])


def _own_norm(s):
    import gaussian_splatting_tile_amd as gs
    case = s["case"]
    kinds = dict(none=gs.BLOCK_NORM_NONE, rms=gs.BLOCK_NORM_RMS, layer=gs.BLOCK_NORM_LAYER)
    gatings = dict(none=gs.BLOCK_GATE_NONE, sigmoid=gs.BLOCK_GATE_SIGMOID, silu=gs.BLOCK_GATE_SILU)
    a = dict(residual=s["residual"], gate=s["gate"], gating=gatings[case["gating"]], scale=s["scale"],
             post=kinds[case["post"]], post_weight=s["post_weight"], post_bias=s["post_bias"],
             pre=kinds[case["pre"]], pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], eps=_EPS)
    out = gs.block_norm_fwd(s["y"], **a)
    out = dict(out=out["out"], **({} if case["pre"] == "none" else dict(norm=out["norm"])))
    if case["mode"] != "train":
        return out
    back = gs.block_norm_bwd(s["y"], s["grad_out"], grad_norm=s["grad_norm"], **a)
    return dict(out, **{k: v for k, v in back.items() if v is not None})


def run(state):
    if state["case"]["op"] == "delta":
        return (_own_delta if own else _plain_delta)(state)
    return (_own_norm if own else _plain_norm)(state)


# ---------------------------------------------------------------- work and exact values

def work(case):
    s = _BYTES[case["dtype"]]
    if case["op"] == "delta":
        B, T, Hk, H, dk, dv = (case[k] for k in ("batch", "steps", "key_heads", "heads", "dk", "dv"))
        rows = B * T * (0.5 if case["ragged"] else 1.0)  # the mean share of the steps that the lengths leave
        qkv, o, gates = rows * (2 * Hk * dk + H * dv) * s, B * T * H * dv * s, rows * H * 8
        state = 2 * B * H * dk * dv * 4
        flops = 7 * rows * H * dk * dv  # S^T k, the decayed sum with the new product, S^T q
        if case["mode"] != "train":
            return {"bytes": qkv + o + gates + state, "flops": flops}
        return {"bytes": 2 * qkv + o + rows * H * dv * s + 2 * gates + B * T * (2 * Hk * dk + H * dv) * s
                + B * T * H * 8 + 2 * state, "flops": 3 * flops}
    N = case["rows"] * case["heads"] * case["width"]
    gate, residual, pre = case["gating"] != "none", case["residual"], case["pre"] != "none"
    read, write = 1 + gate + residual, 1 + pre
    ops = 4 * (case["post"] != "none") + 4 * gate + 2 * case["scale"] + residual + 4 * pre
    if case["mode"] == "train":
        return {"bytes": N * s * (2 * read + write + 1 + pre + read), "flops": 3 * ops * N}
    return {"bytes": N * s * (read + write), "flops": ops * N}


def _exact_delta(s):
    """S_t = a S_{t-1} + k u^T with u = beta (v - a S_{t-1}^T k), o = scale S_t^T q, and their derivatives, step by step."""
    case = s["case"]
    B, T, Hk, H, dk, dv = (case[x] for x in ("batch", "steps", "key_heads", "heads", "dk", "dv"))
    r = H // Hk
    dev = s["q"].device
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=dev)
    live = torch.arange(T, device=dev)[None, :] < n[:, None]
    keep = live.clone() if s["restart"] is None else live & (s["restart"] == 0)
    train, scale = case["mode"] == "train", s["scale"]
    alpha = torch.where(live[..., None], s["log_decay"].double().exp(), 1.0) * torch.where(live & ~keep, 0.0, 1.0)[..., None]
    beta = torch.where(live[..., None], s["beta"].double(), 0.0)
    head = lambda x, t: x[:, t].double().repeat_interleave(r, 1)  # noqa: E731
    mul = lambda S, x: (S * x[..., None]).sum(-2)  # S^T x  # noqa: E731
    outer = lambda x, u: x[..., None] * u[..., None, :]  # noqa: E731

    def step(S, t):
        k, v, b = head(s["k"], t), s["v"][:, t].double(), beta[:, t, :, None]
        S = S * alpha[:, t, :, None, None]
        e = v - mul(S, k)
        return torch.baddbmm(S.reshape(B * H, dk, dv), k.reshape(B * H, dk, 1), (b * e).reshape(B * H, 1, dv)).view_as(S), e, S

    S = s["h0"].double()
    o = torch.zeros((B, T, H, dv), dtype=torch.float64, device=dev)
    marks = []
    for t in range(T):
        if train and t % 64 == 0:
            marks.append(S)
        S = step(S, t)[0]
        o[:, t] = torch.where(live[:, t, None, None], scale * mul(S, head(s["q"], t)), 0.0)
    out = dict(o=o, h_last=S)
    if not train:
        return out
    dS = s["grad_last"].double()
    z = lambda *d: torch.zeros(d, dtype=torch.float64, device=dev)  # noqa: E731
    dq, dk_, dv_, dg, db = z(B, T, Hk, dk), z(B, T, Hk, dk), z(B, T, H, dv), z(B, T, H), z(B, T, H)
    row = lambda S, x: (S * x[..., None, :]).sum(-1)  # S x  # noqa: E731
    for c in range(len(marks) - 1, -1, -1):
        S, states = marks[c], []
        for t in range(64 * c, min(T, 64 * c + 64)):
            before = S
            S, e, decayed = step(S, t)
            states.append((S, e, decayed, before))
        for t in range(min(T, 64 * c + 64) - 1, 64 * c - 1, -1):
            S, e, decayed, before = states[t - 64 * c]
            k, q, b = head(s["k"], t), head(s["q"], t), beta[:, t, :, None]
            on = live[:, t, None, None]
            do = torch.where(on, s["grad_o"][:, t].double(), 0.0)
            dq[:, t] = torch.where(on, scale * row(S, do), 0.0).unflatten(1, (Hk, r)).sum(2)
            dS = dS + outer(torch.where(on, scale * q, 0.0), do)
            du = mul(dS, k)
            de = b * du
            dk_[:, t] = torch.where(on, row(dS, b * e) - row(decayed, de), 0.0).unflatten(1, (Hk, r)).sum(2)
            db[:, t] = torch.where(live[:, t, None], (du * e).sum(-1), 0.0)
            dv_[:, t] = torch.where(on, de, 0.0)
            dS = dS - outer(k, de)
            dg[:, t] = torch.where(live[:, t, None], (dS * before).sum((-1, -2)) * alpha[:, t], 0.0)
            dS = dS * alpha[:, t, :, None, None]
    return dict(out, grad_q=dq, grad_k=dk_, grad_v=dv_, grad_log_decay=dg, grad_beta=db, grad_h0=dS)


def _exact_norm(s):
    case = s["case"]
    train = case["mode"] == "train"
    names = ["y", "gate", "residual", "post_weight", "post_bias", "scale", "pre_weight", "pre_bias"]
    a = {k: None if s[k] is None else s[k].double().clone().requires_grad_(train) for k in names}

    def one(x, kind, weight, bias):
        if kind == "rms":
            return weight * x / torch.sqrt(torch.mean(x * x, -1, keepdim=True) + _EPS)
        m = torch.mean(x, -1, keepdim=True)
        return weight * (x - m) / torch.sqrt(torch.mean((x - m) ** 2, -1, keepdim=True) + _EPS) + bias

    x = a["y"]
    if case["post"] != "none":
        x = one(x, case["post"], a["post_weight"], a["post_bias"])
    if case["gating"] != "none":
        x = x / (1 + torch.exp(-a["gate"])) * (a["gate"] if case["gating"] == "silu" else 1.0)
    if a["scale"] is not None:
        x = x * a["scale"]
    if a["residual"] is not None:
        x = x + a["residual"]
    out = dict(out=x)
    if case["pre"] != "none":
        out["norm"] = one(x, case["pre"], a["pre_weight"], a["pre_bias"])
    if train:
        up = [s["grad_out"].double()] + ([s["grad_norm"].double()] if case["pre"] != "none" else [])
        leaves = [k for k in names if a[k] is not None]
        got = torch.autograd.grad(list(out.values()), [a[k] for k in leaves], up)
        out = {k: v.detach() for k, v in out.items()}
        out.update({"grad_" + k: v for k, v in zip(leaves, got)})
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_delta(s) if case["op"] == "delta" else _exact_norm(s)
