"""Binding of the calls of libgs that make up a recurrent block of a network:
the gated delta rule (gs_delta_rule_fwd / gs_delta_rule_bwd) and the norms
around a block with its gate, residual scale and residual
(gs_block_norm_fwd / gs_block_norm_bwd). As in training.py, torch supplies
device memory and the current HIP stream; the work is libgs's kernels.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import (GS_BLOCK_GATE_NONE, GS_BLOCK_GATE_SIGMOID, GS_BLOCK_GATE_SILU, GS_BLOCK_NORM_LAYER,
                   GS_BLOCK_NORM_NONE, GS_BLOCK_NORM_RMS, GS_DELTA_CHUNK, GS_DELTA_FEW)
from .training import _TYPES, _dtype, _elsewhere, _launch, _on, _ptr, _stream

BLOCK_NORM_NONE, BLOCK_NORM_RMS, BLOCK_NORM_LAYER = GS_BLOCK_NORM_NONE, GS_BLOCK_NORM_RMS, GS_BLOCK_NORM_LAYER
BLOCK_GATE_NONE, BLOCK_GATE_SIGMOID, BLOCK_GATE_SILU = GS_BLOCK_GATE_NONE, GS_BLOCK_GATE_SIGMOID, GS_BLOCK_GATE_SILU


_MOST = 1 << 30  # what the library takes along a dimension; more would not fit the fields of a description


# ---------------------------------------------------------------- the delta rule

def _strided(t, shape, dtype, name, device):
    """The address of a tensor of device number `device` with this shape and type, and contiguous last dimension."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise TypeError(f"{name} must be a tensor on cuda:{device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous() and shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return t.data_ptr()


def _delta(q, k, v, log_decay, beta, scale, lengths, restart):
    """The C description of a call, the addresses of its inputs, and its sizes."""
    shape, vshape, n, t = q.shape, v.shape, q.get_device(), q.dtype
    if len(shape) != 4 or len(vshape) != 4:
        raise ValueError("q, k and v must be [B, T, heads, dim]")
    if n < 0:
        raise TypeError("q, k and v must be device tensors")
    if max(shape) > _MOST or max(vshape) > _MOST:
        raise ValueError(f"q, k and v may have at most {_MOST} elements along a dimension")
    B, T, Hk, dk = shape
    H, dv = vshape[2:]
    gates, f32 = (B, T, H), torch.float32
    code = _dtype(q, "q, k and v")
    p = (_strided(q, shape, t, "q", n), _strided(k, shape, t, "k", n), _strided(v, (B, T, H, dv), t, "v", n),
         _strided(log_decay, gates, f32, "log_decay", n), _strided(beta, gates, f32, "beta", n))
    r = _lib.GsDeltaRule(code, B, T, Hk, H, dk, dv, dk ** -0.5 if scale is None else scale, *q.stride()[:3],
                         *k.stride()[:3], *v.stride()[:3], *log_decay.stride()[:2], *beta.stride()[:2],
                         None if lengths is None else _ptr(lengths, (B,), torch.int32, "lengths", n),
                         None if restart is None else _ptr(restart, (B, T), torch.uint8, "restart", n))
    return r, p, (B, T, Hk, H, dk, dv)


def _scratch(need, scratch, device):
    """The workspace's tensor (kept until the call is enqueued), address and size."""
    if not need:
        return None, None, 0
    if scratch is None:
        scratch = torch.empty((need,), dtype=torch.uint8, device=device)
    return scratch, _ptr(scratch, None, None, "scratch", device.index), scratch.numel() * scratch.element_size()


def delta_rule_scratch_bytes(batch: int, steps: int, heads: int, key_dim: int, value_dim: int, backward=False,
                             dtype=torch.float32, key_heads=None) -> int:
    """Bytes of the workspace delta_rule_fwd (or delta_rule_bwd) takes for this shape; without `key_heads`, bytes that
    are enough for any number of them."""
    r = _lib.GsDeltaRule()
    r.batch, r.steps, r.heads = int(batch), int(steps), int(heads)
    r.key_heads = r.heads if key_heads is None else int(key_heads)
    r.key_dim, r.value_dim, r.dtype = int(key_dim), int(value_dim), _dtype(torch.empty(0, dtype=dtype), "dtype")
    return int(_lib.load().gs_delta_rule_scratch_bytes(ctypes.byref(r), int(bool(backward))))


def delta_rule_ckpt_rows(steps: int) -> int:
    """Checkpoint rows of a sequence: the states in front of steps 64, 128, ... below `steps`."""
    return max(0, -(-int(steps) // GS_DELTA_CHUNK) - 1)


def delta_rule_fwd(q, k, v, log_decay, beta, h0=None, scale=None, lengths=None, restart=None, checkpoints=False,
                   out=None, scratch=None, stream=None):
    """gs_delta_rule_fwd: S_t = a_t S_{t-1} + k_t u_t^T with u_t = beta_t (v_t - a_t S_{t-1}^T k_t), a_t =
    exp(log_decay_t), and o_t = scale S_t^T q_t, along dim 1. q, k [B, T, Hk, dk] and v [B, T, H, dv] of one type
    (float32, bfloat16 or float16; any strides but contiguous dims), H a multiple of Hk (head h uses key head
    h // (H // Hk)), dk and dv at most 128; log_decay and beta float32 [B, T, H]; scale dk ** -0.5 unless given.
    h0 float32 [B, H, dk, dv]; lengths int32 [B]; restart uint8 [B, T]. Returns dict o [B, T, H, dv], h_last float32
    [B, H, dk, dv] and ckpt (float32 [B, delta_rule_ckpt_rows(T), H, dk, dv] with checkpoints, for delta_rule_bwd;
    else None). `out` may give any of them; out["h_last"] may be h0 itself (one state buffer for serving), no other
    output may overlap an input or another output. Past 8 steps a step's stride in q, k and v is at most 2 ** 22. With `stream` (not the current one) the call allocates and runs on it: order it
    behind whatever wrote the inputs, and the use of what it returns behind it. Calls that share a `scratch` must
    not overlap."""
    if stream is not None and _elsewhere(stream, q.device):
        return _on(stream, lambda: delta_rule_fwd(q, k, v, log_decay, beta, h0, scale, lengths, restart, checkpoints,
                                                  out, scratch), out)
    lib = _lib.load()
    r, p, (B, T, Hk, H, dk, dv) = _delta(q, k, v, log_decay, beta, scale, lengths, restart)
    dev, f32, state = q.device, torch.float32, (B, H, dk, dv)
    n = dev.index
    o = h_last = ckpt = pc = None
    if out is not None:
        o, h_last, ckpt = out.get("o"), out.get("h_last"), out.get("ckpt")
    if o is None:
        o = q.new_empty((B, T, H, dv))
        po = o.data_ptr()
    else:
        po = _ptr(o, (B, T, H, dv), q.dtype, "o", n)
    if h_last is None:
        h_last = q.new_empty(state, dtype=f32)
        pl = h_last.data_ptr()
    else:
        pl = _ptr(h_last, state, f32, "h_last", n)
    if checkpoints or ckpt is not None:
        rows = (B, delta_rule_ckpt_rows(T), H, dk, dv)
        if ckpt is None:
            ckpt = q.new_empty(rows, dtype=f32)
        pc = _ptr(ckpt, rows, f32, "ckpt", n)
    ph, ps, nbytes = _ptr(h0, state, f32, "h0", n), None, 0
    if T > GS_DELTA_FEW:
        scratch, ps, nbytes = _scratch(int(lib.gs_delta_rule_scratch_bytes(ctypes.byref(r), 0)), scratch, dev)
    _launch(dev, lib.gs_delta_rule_fwd, ctypes.byref(r), *p, ph, po, pl, pc, ps, nbytes, _stream(stream, dev))
    return dict(o=o, h_last=h_last, ckpt=ckpt)


def delta_rule_bwd(q, k, v, log_decay, beta, grad_o, h0=None, ckpt=None, grad_last=None, scale=None, lengths=None,
                   restart=None, out=None, scratch=None, stream=None):
    """gs_delta_rule_bwd: gradients of delta_rule_fwd, which gave `ckpt` (needed when T > 64). grad_o [B, T, H, dv] of
    v's type; grad_last float32 [B, H, dk, dv] or None. Returns dict grad_q, grad_k [B, T, Hk, dk] (summed over the
    heads of a key head), grad_v [B, T, H, dv], grad_log_decay, grad_beta float32 [B, T, H], grad_h0 float32
    [B, H, dk, dv]. `out` may give all of them (grad_h0 or not). `stream` and `scratch` as for delta_rule_fwd."""
    if stream is not None and _elsewhere(stream, q.device):
        return _on(stream, lambda: delta_rule_bwd(q, k, v, log_decay, beta, grad_o, h0, ckpt, grad_last, scale,
                                                  lengths, restart, out, scratch), out)
    lib = _lib.load()
    r, p, (B, T, Hk, H, dk, dv) = _delta(q, k, v, log_decay, beta, scale, lengths, restart)
    dev, f32, t, state = q.device, torch.float32, q.dtype, (B, H, dk, dv)
    n, keys, values, gates = dev.index, (B, T, Hk, dk), (B, T, H, dv), (B, T, H)
    if out is None:
        e = q.new_empty
        out = dict(grad_q=e(keys), grad_k=e(keys), grad_v=e(values), grad_log_decay=e(gates, dtype=f32),
                   grad_beta=e(gates, dtype=f32), grad_h0=e(state, dtype=f32))
    p += (_ptr(h0, state, f32, "h0", n), _ptr(ckpt, (B, delta_rule_ckpt_rows(T), H, dk, dv), f32, "ckpt", n),
          _ptr(grad_o, values, t, "grad_o", n), _ptr(grad_last, state, f32, "grad_last", n),
          _ptr(out["grad_q"], keys, t, "grad_q", n), _ptr(out["grad_k"], keys, t, "grad_k", n),
          _ptr(out["grad_v"], values, t, "grad_v", n), _ptr(out["grad_log_decay"], gates, f32, "grad_log_decay", n),
          _ptr(out["grad_beta"], gates, f32, "grad_beta", n), _ptr(out.get("grad_h0"), state, f32, "grad_h0", n))
    scratch, ps, nbytes = _scratch(int(lib.gs_delta_rule_scratch_bytes(ctypes.byref(r), 1)), scratch, dev)
    _launch(dev, lib.gs_delta_rule_bwd, ctypes.byref(r), *p, ps, nbytes, _stream(stream, dev))
    return out


# ---------------------------------------------------------------- the norms around a block

def _breaks(t):
    """The places between leading dimensions of t where its rows do not follow at one stride, and the sizes and strides
    of its dimensions that have more than one element."""
    dims = [(i, n, s) for i, (n, s) in enumerate(zip(t.shape[:-1], t.stride()[:-1])) if n > 1]
    return {b[0] for a, b in zip(dims, dims[1:]) if a[2] != b[1] * b[2]}


def _row_strides(t, at):
    """(outer, inner) strides of t's rows, the leading dimensions from `at` on being the inner ones."""
    outer = [s for n, s in zip(t.shape[:at], t.stride()[:at]) if n > 1]
    inner = [s for n, s in zip(t.shape[at:-1], t.stride()[at:-1]) if n > 1]
    return outer[-1] if outer else 0, inner[-1] if inner else 0


def _norm_call(y, gate, residual, gating, scale, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps):
    """The C description of a call and the addresses of its inputs."""
    shape, t, n = y.shape, y.dtype, y.get_device()
    if len(shape) < 2:
        raise ValueError("y must be [..., width]")
    if n < 0:
        raise TypeError("y must be a device tensor")
    D = shape[-1]
    if not 0 < D <= _MOST:
        raise ValueError(f"a row of y must have 1 to {_MOST} elements")
    p = [_strided(y, shape, t, "y", n), None if gate is None else _strided(gate, shape, t, "gate", n),
         None if residual is None else _strided(residual, shape, t, "residual", n)]
    outer, inner = y.numel() // D, 1
    if y.is_contiguous() and (gate is None or gate.is_contiguous()) and (residual is None or residual.is_contiguous()):
        strides = (D, 0, D, 0, D, 0)
    else:
        rows = [x for x in (y, gate, residual) if x is not None]
        cuts = set().union(*(_breaks(x) for x in rows))
        if len(cuts) > 1:
            raise ValueError("the rows of y, gate and residual must follow at one stride, or at two that break at the "
                             "same dimension")
        at = cuts.pop() if cuts else len(shape) - 1
        for m in shape[at:-1]:
            inner *= m
        outer = outer // inner if inner else 0
        if inner > _MOST:
            raise ValueError(f"y, gate and residual may have at most {_MOST} rows")
        strides = []
        for x in (y, gate, residual):
            strides += (0, 0) if x is None else _row_strides(x, at)
    wt, wide = None, (D,)
    for w, name in ((post_weight, "post_weight"), (post_bias, "post_bias"), (scale, "scale"),
                    (pre_weight, "pre_weight"), (pre_bias, "pre_bias")):
        if w is None:
            p.append(None)
        else:
            if wt is None:
                wt = w.dtype
            p.append(_ptr(w, wide, wt, name, n))
    d = _lib.GsBlockNorm(_dtype(y, "y"), _lib.GS_F32 if wt is None else _TYPES.get(wt, -1), post, gating, pre,
                         inner or 1, D, eps, outer, *strides)
    return d, p


def block_norm_fwd(y, residual=None, gate=None, gating=BLOCK_GATE_NONE, scale=None, post=BLOCK_NORM_NONE,
                   post_weight=None, post_bias=None, pre=BLOCK_NORM_NONE, pre_weight=None, pre_bias=None, eps=1e-6,
                   want_out=True, out=None, stream=None):
    """gs_block_norm_fwd: what lies between a block and the next one, over the rows (last dimension, at most 16384
    elements) of y: t = post norm of y (weight, bias), out = residual + scale act(gate) t, norm = pre norm of out
    (weight, bias). Norms: BLOCK_NORM_NONE, BLOCK_NORM_RMS, BLOCK_NORM_LAYER; gating: BLOCK_GATE_NONE,
    BLOCK_GATE_SIGMOID, BLOCK_GATE_SILU. y, gate, residual [..., width] of one shape and type (float32, bfloat16 or
    float16), rows at any one stride, or two (tokens and heads of a part of a projection); weights, biases and scale
    [width], all float32 or all of y's type. Returns dict out (None unless want_out) and norm (None without pre). `out` may give them;
    out["out"] may be y, gate or residual itself. `stream` as for delta_rule_fwd."""
    if stream is not None and _elsewhere(stream, y.device):
        return _on(stream, lambda: block_norm_fwd(y, residual, gate, gating, scale, post, post_weight, post_bias, pre,
                                                  pre_weight, pre_bias, eps, want_out, out), out)
    lib = _lib.load()
    d, p = _norm_call(y, gate, residual, gating, scale, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps)
    dev = y.device
    x = norm = px = pn = None
    if out is not None:
        x, norm = out.get("out"), out.get("norm")
    if x is not None:
        px = _ptr(x, y.shape, y.dtype, "out", dev.index)
    elif want_out:
        x = y.new_empty(y.shape)
        px = x.data_ptr()
    if pre == BLOCK_NORM_NONE:
        norm = None
    elif norm is not None:
        pn = _ptr(norm, y.shape, y.dtype, "norm", dev.index)
    else:
        norm = y.new_empty(y.shape)
        pn = norm.data_ptr()
    _launch(dev, lib.gs_block_norm_fwd, ctypes.byref(d), *p, px, pn, _stream(stream, dev))
    return dict(out=x, norm=norm)


def block_norm_bwd(y, grad_out, grad_norm=None, residual=None, gate=None, gating=BLOCK_GATE_NONE, scale=None,
                   post=BLOCK_NORM_NONE, post_weight=None, post_bias=None, pre=BLOCK_NORM_NONE, pre_weight=None,
                   pre_bias=None, eps=1e-6, out=None, scratch=None, stream=None):
    """gs_block_norm_bwd: gradients of block_norm_fwd from grad_out (None: zero, only with pre) and grad_norm (with
    pre). Returns dict grad_y, grad_gate, grad_residual (rows), grad_post_weight, grad_post_bias, grad_scale,
    grad_pre_weight, grad_pre_bias (float32 [width], sums over the rows); None for what the call does not have.
    `out` may give them (those it lacks of gate, residual and the sums are not computed); grad_y, grad_gate and
    grad_residual may each be grad_out or grad_norm itself. `stream` as for delta_rule_fwd; calls that share a
    `scratch` must not overlap."""
    if stream is not None and _elsewhere(stream, y.device):
        return _on(stream, lambda: block_norm_bwd(y, grad_out, grad_norm, residual, gate, gating, scale, post,
                                                  post_weight, post_bias, pre, pre_weight, pre_bias, eps, out,
                                                  scratch), out)
    lib = _lib.load()
    d, p = _norm_call(y, gate, residual, gating, scale, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps)
    dev, shape, t, f32 = y.device, y.shape, y.dtype, torch.float32
    n, wide = dev.index, shape[-1:]
    rows = (("grad_y", y), ("grad_gate", None if gating == BLOCK_GATE_NONE else gate), ("grad_residual", residual))
    sums = (("grad_post_weight", post_weight), ("grad_post_bias", post_bias), ("grad_scale", scale),
            ("grad_pre_weight", pre_weight), ("grad_pre_bias", pre_bias))
    p += [_ptr(grad_out, shape, t, "grad_out", n), _ptr(grad_norm, shape, t, "grad_norm", n)]
    if out is None:
        out, ps = {}, []
        for k, x in rows:
            out[k] = None if x is None else y.new_empty(shape)
            p.append(None if x is None else out[k].data_ptr())
        for k, w in sums:
            out[k] = None if w is None else y.new_empty(wide, dtype=f32)
            ps.append(None if w is None else out[k].data_ptr())
    else:
        p += [_ptr(out["grad_y"], shape, t, "grad_y", n), _ptr(out.get("grad_gate"), shape, t, "grad_gate", n),
              _ptr(out.get("grad_residual"), shape, t, "grad_residual", n)]
        ps = [_ptr(out.get(k), wide, f32, k, n) for k, _ in sums]
    need = int(lib.gs_block_norm_scratch_bytes(ctypes.byref(d))) if any(ps) else 0
    scratch, pw, nbytes = _scratch(need, scratch, dev)
    _launch(dev, lib.gs_block_norm_bwd, ctypes.byref(d), *p, *ps, pw, nbytes, _stream(stream, dev))
    return out
