"""Binding of the sequence and training calls of libgs: the gated linear
recurrence (gs_recurrence_fwd / gs_recurrence_bwd), the global gradient norm
and clipping (gs_grad_norm, gs_clip_grads) and the Adam update with that
clipping (gs_adam_step). As in rasterizer.py, torch supplies device memory
and the current HIP stream; the work is libgs's kernels.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import GS_ADAM_SKIP_NONFINITE, GS_GATE_LINEAR, GS_GATE_SIGMOID, GS_NORM_L2, GS_NORM_MAX

GATE_LINEAR, GATE_SIGMOID = GS_GATE_LINEAR, GS_GATE_SIGMOID
NORM_L2, NORM_MAX = GS_NORM_L2, GS_NORM_MAX
_TYPES = {torch.float32: _lib.GS_F32, torch.bfloat16: _lib.GS_BF16, torch.float16: _lib.GS_F16}


# A call's own time on the host counts where a step is a few microseconds of
# GPU work: pointers are passed as plain integers and checked with the
# cheapest tensor attributes that say what is needed.

def _stream(stream, device):
    """The raw handle of `stream`, or of the device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def _of_device(stream, device):
    if stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors are on {device}")


def _on(stream, call, given=None):
    """call() with `stream` current, so that what it allocates is ordered with what it launches
    there. Tensors that it returns (other than those of the dict `given`) may be used and
    dropped on the caller's stream, once that is ordered behind `stream`: their memory is not
    handed out again before the caller's work on them."""
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = call()
    given = [] if given is None else [id(t) for t in given.values()]
    for t in out.values() if isinstance(out, dict) else [out]:
        if t is not None and id(t) not in given:
            t.record_stream(caller)
    return out


def _elsewhere(stream, device):
    """Whether a call on `device` is asked to run on another stream than the current one."""
    if stream is None:
        return False
    _of_device(stream, device)
    return stream.cuda_stream != torch.cuda.current_stream(device).cuda_stream


def _launch(device, call, *args):
    """A library call that launches: with the tensors' device current."""
    if torch._C._cuda_getDevice() == device.index:
        _lib.check(call(*args))
    else:
        with torch.cuda.device(device):
            _lib.check(call(*args))


class _Held:
    """Tensors that an object made on the stream of its construction and uses on others too."""

    def _hold(self, tensors):
        self._held, self._streams = tensors, {_stream(None, self.device)}

    def _call_stream(self, stream):
        """The raw handle of a call's stream. The tensors are not handed out again before the work on it is done."""
        if stream is not None:
            _of_device(stream, self.device)
        raw = _stream(stream, self.device)
        if raw not in self._streams:
            for t in self._held:
                t.record_stream(torch.cuda.current_stream(self.device) if stream is None else stream)
            self._streams.add(raw)
        return raw


def _ptr(t, shape, dtype, name, device):
    """The address of a contiguous tensor of device number `device`, of this shape (None: any)
    and type (None: any)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise TypeError(f"{name} must be a tensor on cuda:{device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dtype(t, name):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return code


def _recurrence(gate, x, gating, lengths, restart):
    """The C description of a call, and its sizes."""
    shape = gate.shape
    if len(shape) != 3 or x.shape != shape or x.dtype != gate.dtype or x.device != gate.device:
        raise ValueError("gate and x must be [B, T, D] of the same shape, type and device")
    if not gate.is_cuda:
        raise TypeError("gate and x must be device tensors")
    B, T, D = shape
    index = gate.get_device()
    gb, gt, gd = gate.stride()
    xb, xt, xd = x.stride()
    if D > 1 and (gd != 1 or xd != 1):
        raise ValueError("gate and x must have contiguous channels (last stride 1)")
    r = _lib.GsRecurrence(_dtype(gate, "gate and x"), int(gating), B, T, D, gb, gt, xb, xt,
                          _ptr(lengths, (B,), torch.int32, "lengths", index),
                          _ptr(restart, (B, T), torch.uint8, "restart", index))
    return r, B, T, D


def _scratch(lib, r, scratch, device):
    """The workspace's tensor (kept until the call is enqueued), address and size."""
    if r.steps <= _lib.GS_RECURRENCE_CHUNK:
        return None, None, 0
    if scratch is None:
        need = int(lib.gs_recurrence_scratch_bytes(ctypes.byref(r)))
        scratch = torch.empty((need,), dtype=torch.uint8, device=device)
    return scratch, _ptr(scratch, None, None, "scratch", device.index), scratch.numel() * scratch.element_size()


def recurrence_scratch_bytes(batch: int, steps: int, channels: int) -> int:
    """Bytes of the workspace recurrence_fwd and recurrence_bwd take for this shape."""
    r = _lib.GsRecurrence()
    r.batch, r.steps, r.channels = int(batch), int(steps), int(channels)
    return int(_lib.load().gs_recurrence_scratch_bytes(ctypes.byref(r)))


def recurrence_ckpt_rows(steps: int) -> int:
    """Checkpoint rows of a sequence: the states in front of steps 128, 256, ... below `steps`."""
    return max(0, -(-int(steps) // _lib.GS_RECURRENCE_CHUNK) - 1)


def recurrence_fwd(gate, x, h0=None, gating=GATE_LINEAR, lengths=None, restart=None, checkpoints=False, out=None,
                   scratch=None, stream=None):
    """gs_recurrence_fwd: h_t = a_t h_{t-1} + u_t along dim 1 of gate and x ([B, T, D], float32,
    bfloat16 or float16; any batch and step strides, contiguous channels). gating: GATE_LINEAR
    (a = gate, u = x) or GATE_SIGMOID (a = sigmoid(gate), u = (1 - a) x). h0 float32 [B, D];
    lengths int32 [B]; restart uint8 [B, T]. Returns dict h [B, T, D], h_last float32 [B, D] and
    ckpt (float32 [B, recurrence_ckpt_rows(T), D] with checkpoints, for recurrence_bwd; else
    None). `out` may give any of them; out["h_last"] may be h0 itself (one state buffer for
    step-by-step serving, T = 1), no other output may overlap an input. With `stream` (not the
    current one) the call allocates and runs on it: order it behind whatever wrote the inputs,
    and the use of what it returns behind it. Calls that share a `scratch` must not overlap."""
    if _elsewhere(stream, gate.device):
        return _on(stream, lambda: recurrence_fwd(gate, x, h0, gating, lengths, restart, checkpoints, out, scratch), out)
    lib = _lib.load()
    r, B, T, D = _recurrence(gate, x, gating, lengths, restart)
    dev, f32, whole, state = gate.device, torch.float32, (B, T, D), (B, D)
    n = dev.index
    h = h_last = ckpt = None
    if out is not None:
        h, h_last, ckpt = out.get("h"), out.get("h_last"), out.get("ckpt")
    if h is None:
        h = gate.new_empty(whole)
        ph = h.data_ptr()
    else:
        ph = _ptr(h, whole, gate.dtype, "h", n)
    if h_last is None:
        h_last = gate.new_empty(state, dtype=f32)
        pl = h_last.data_ptr()
    else:
        pl = _ptr(h_last, state, f32, "h_last", n)
    if ckpt is None and checkpoints:
        ckpt = gate.new_empty((B, recurrence_ckpt_rows(T), D), dtype=f32)
    scratch, ps, nbytes = _scratch(lib, r, scratch, dev)
    _launch(
        dev, lib.gs_recurrence_fwd, ctypes.byref(r), gate.data_ptr(), x.data_ptr(), _ptr(h0, state, f32, "h0", n), ph,
        pl, None if ckpt is None else _ptr(ckpt, (B, recurrence_ckpt_rows(T), D), f32, "ckpt", n), ps, nbytes,
        _stream(stream, dev))
    return dict(h=h, h_last=h_last, ckpt=ckpt)


def recurrence_bwd(gate, x, grad_h, h0=None, ckpt=None, grad_last=None, gating=GATE_LINEAR, lengths=None,
                   restart=None, out=None, scratch=None, stream=None):
    """gs_recurrence_bwd: gradients of recurrence_fwd, which gave `ckpt` (needed when T > 128).
    grad_h [B, T, D] of gate's type; grad_last float32 [B, D] or None. Returns dict grad_gate,
    grad_x [B, T, D], grad_h0 float32 [B, D]. `stream` and `scratch` as for recurrence_fwd."""
    if _elsewhere(stream, gate.device):
        return _on(stream, lambda: recurrence_bwd(gate, x, grad_h, h0, ckpt, grad_last, gating, lengths, restart, out,
                                                  scratch), out)
    lib = _lib.load()
    r, B, T, D = _recurrence(gate, x, gating, lengths, restart)
    dev, f32, t, whole, state = gate.device, torch.float32, gate.dtype, (B, T, D), (B, D)
    n = dev.index
    if out is None:
        out = dict(grad_gate=gate.new_empty(whole), grad_x=gate.new_empty(whole),
                   grad_h0=gate.new_empty(state, dtype=f32))
    scratch, ps, nbytes = _scratch(lib, r, scratch, dev)
    _launch(
        dev, lib.gs_recurrence_bwd, ctypes.byref(r), gate.data_ptr(), x.data_ptr(), _ptr(h0, state, f32, "h0", n),
        None if ckpt is None else _ptr(ckpt, (B, recurrence_ckpt_rows(T), D), f32, "ckpt", n),
        _ptr(grad_h, whole, t, "grad_h", n), _ptr(grad_last, state, f32, "grad_last", n),
        _ptr(out["grad_gate"], whole, t, "grad_gate", n), _ptr(out["grad_x"], whole, t, "grad_x", n),
        _ptr(out.get("grad_h0"), state, f32, "grad_h0", n), ps, nbytes, _stream(stream, dev))
    return out


def _device_of(tensors, name):
    if not tensors:
        raise ValueError(f"{name}: the list is empty")
    dev = tensors[0].device
    if dev.type != "cuda" or any(t.device != dev for t in tensors):
        raise TypeError(f"{name} must be tensors of one device")
    return dev


class GradList(_Held):
    """A list of gradients (float32, bfloat16 or float16, each contiguous, types mixed as
    wanted) whose global norm is taken and clipped. Holds the tensors, their description for
    the C call and the workspace, so a step's call only launches. Clipping writes to `out`
    (default: in place). Calls of one list share its workspace and must not overlap; on another
    stream than that of the construction they are ordered behind it by the caller."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        self.device = _device_of(self.grads, "grads")
        if len(self.out) != len(self.grads):
            raise ValueError("out must hold one tensor for each gradient")
        self._n = len(self.grads)
        self._list = (_lib.GsGradTensor * self._n)()
        n = self.device.index
        for d, g, o in zip(self._list, self.grads, self.out):
            if o.shape != g.shape:
                raise ValueError("out must have the shapes of grads")
            d.grad, d.out = _ptr(g, None, None, "grad", n), _ptr(o, None, g.dtype, "out", n)
            d.count, d.dtype = g.numel(), _dtype(g, "grad")
        self._lib = _lib.load()
        self.scratch = torch.empty((int(self._lib.gs_grad_scratch_bytes()),), dtype=torch.uint8, device=self.device)
        self._pscratch = self.scratch.data_ptr()
        self._hold([self.scratch])

    def _norm(self, out):
        if out is not None:
            return out, _ptr(out, (), torch.float32, "out", self.device.index)
        out = torch.empty((), dtype=torch.float32, device=self.device)
        return out, out.data_ptr()

    def norm(self, kind=NORM_L2, out=None, stream=None):
        """gs_grad_norm: the global norm, a float32 tensor of no dimensions on the device."""
        if out is None and _elsewhere(stream, self.device):
            return _on(stream, lambda: self.norm(kind))
        out, po = self._norm(out)
        _launch(self.device, self._lib.gs_grad_norm, self._list, self._n, int(kind), po, self._pscratch,
                self._call_stream(stream))
        return out

    def clip(self, max_norm, kind=NORM_L2, out=None, stream=None):
        """gs_clip_grads: scales by min(1, max_norm / (norm + 1e-6)); returns the norm before."""
        if out is None and _elsewhere(stream, self.device):
            return _on(stream, lambda: self.clip(max_norm, kind))
        out, po = self._norm(out)
        _launch(self.device, self._lib.gs_clip_grads, self._list, self._n, int(kind), float(max_norm), po,
                self._pscratch, self._call_stream(stream))
        return out


def grad_norm(grads, kind=NORM_L2, stream=None):
    """The global norm of a list of gradients (GradList(grads).norm())."""
    grads = list(grads)
    if stream is not None and _elsewhere(stream, _device_of(grads, "grads")):
        return _on(stream, lambda: grad_norm(grads, kind))
    return GradList(grads).norm(kind)


def clip_grads(grads, max_norm, kind=NORM_L2, out=None, stream=None):
    """Clips a list of gradients by their global norm, in place or into `out`; returns the norm."""
    grads = list(grads)
    if stream is not None and _elsewhere(stream, _device_of(grads, "grads")):
        return _on(stream, lambda: clip_grads(grads, max_norm, kind, out))
    return GradList(grads, out).clip(max_norm, kind)


class Adam(_Held):
    """gs_adam_step over a fixed list of parameters and gradient buffers: Adam with decoupled
    weight decay, the gradients clipped on the way by their global norm (max_norm > 0). lr and
    weight_decay are numbers or one number per tensor (`set_lr` changes them); the moments
    (exp_avg, exp_avg_sq, float32) start at 0 and the device step counter at `step` unless
    given. With skip_nonfinite a step whose gradients hold an infinity or a NaN changes
    nothing. Steps of one object must not overlap; on another stream than that of the
    construction they are ordered behind it by the caller."""

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, max_norm=0.0,
                 skip_nonfinite=False, exp_avg=None, exp_avg_sq=None, step=0):
        self.params, self.grads = list(params), list(grads)
        self.device = dev = _device_of(self.params + self.grads, "params and grads")
        n = self._n = len(self.params)
        if len(self.grads) != n:
            raise ValueError("params and grads must be lists of one length")
        f32 = torch.float32
        zeros = lambda: [torch.zeros(p.shape, dtype=f32, device=dev) for p in self.params]
        self.exp_avg = zeros() if exp_avg is None else list(exp_avg)
        self.exp_avg_sq = zeros() if exp_avg_sq is None else list(exp_avg_sq)
        if len(self.exp_avg) != n or len(self.exp_avg_sq) != n:
            raise ValueError("exp_avg and exp_avg_sq must hold one tensor for each parameter")
        if step < 0:
            raise ValueError("step counts the updates taken before: it is not negative")
        self.steps = torch.full((1,), int(step), dtype=torch.int64, device=dev)
        self.norm = torch.zeros((), dtype=f32, device=dev)
        self._cfg = _lib.GsAdam(float(betas[0]), float(betas[1]), float(eps), float(max_norm),
                                GS_ADAM_SKIP_NONFINITE if skip_nonfinite else 0)
        self._want_norm = max_norm > 0 or skip_nonfinite
        self._list = (_lib.GsAdamTensor * n)()
        for d, p, g, m, v in zip(self._list, self.params, self.grads, self.exp_avg, self.exp_avg_sq):
            if g.shape != p.shape or m.shape != p.shape or v.shape != p.shape:
                raise ValueError("a gradient or moment does not have its parameter's shape")
            d.param, d.grad = _ptr(p, None, None, "param", dev.index), _ptr(g, None, None, "grad", dev.index)
            d.m, d.v = _ptr(m, None, f32, "exp_avg", dev.index), _ptr(v, None, f32, "exp_avg_sq", dev.index)
            d.count, d.param_dtype, d.grad_dtype = p.numel(), _dtype(p, "param"), _dtype(g, "grad")
        self.set_lr(lr)
        for d, wd in zip(self._list, self._each(weight_decay, "weight_decay")):
            d.weight_decay = wd
        self._lib = _lib.load()
        self.scratch = torch.empty((int(self._lib.gs_grad_scratch_bytes()),), dtype=torch.uint8, device=dev)
        self._fixed = (ctypes.byref(self._cfg), self._list, n, self.steps.data_ptr(),
                       self.norm.data_ptr() if self._want_norm else None, self.scratch.data_ptr())
        self._hold([self.scratch, self.steps, self.norm] + (self.exp_avg if exp_avg is None else []) +
                   (self.exp_avg_sq if exp_avg_sq is None else []))

    def _each(self, v, name):
        v = [float(v)] * self._n if isinstance(v, (int, float)) else [float(x) for x in v]
        if len(v) != self._n:
            raise ValueError(f"{name} must be a number or one number for each parameter")
        return v

    def set_lr(self, lr):
        """The learning rate (or one for each tensor) of the steps that follow."""
        for d, v in zip(self._list, self._each(lr, "lr")):
            d.lr = v

    def step(self, stream=None):
        """One update. Returns the gradients' global norm before clipping (a device tensor that
        the next step overwrites), or None when nothing asks for it."""
        _launch(self.device, self._lib.gs_adam_step, *self._fixed, self._call_stream(stream))
        return self.norm if self._want_norm else None
