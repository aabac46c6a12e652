"""Tensors and streams of different devices are refused by the sequence and training calls,
before anything is launched. Needs no GPU: the tensors only say that they are on one."""
from types import SimpleNamespace

import pytest
import torch


class On(torch.Tensor):
    """A host tensor that says it is on cuda:`index`."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


def on(index, *shape, dtype=torch.float32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.index = index
    return t


STREAM = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=12345)


def test_recurrence_refuses_other_devices():
    import gaussian_splatting_tile_amd as gs
    B, T, D = 2, 100, 8
    x = on(0, B, T, D)
    given = lambda i: dict(h=on(i, B, T, D), h_last=on(i, B, D), ckpt=on(i, B, 0, D))
    for bad in (1, -1):
        for kw in (dict(h0=on(bad, B, D)), dict(lengths=on(bad, B, dtype=torch.int32)),
                   dict(restart=on(bad, B, T, dtype=torch.uint8)), dict(out=dict(given(0), h=on(bad, B, T, D))),
                   dict(out=dict(given(0), h_last=on(bad, B, D))), dict(out=dict(given(0), ckpt=on(bad, B, 0, D)))):
            with pytest.raises(TypeError, match="cuda:0"):
                gs.recurrence_fwd(x, x, **kw)
        back = lambda i: dict(grad_gate=on(i, B, T, D), grad_x=on(i, B, T, D), grad_h0=on(i, B, D))
        for kw in (dict(grad_h=on(bad, B, T, D)), dict(h0=on(bad, B, D)), dict(grad_last=on(bad, B, D)),
                   dict(ckpt=on(bad, B, 0, D)), dict(lengths=on(bad, B, dtype=torch.int32)),
                   *[dict(out=dict(back(0), **{k: v})) for k, v in back(bad).items()]):
            with pytest.raises(TypeError, match="cuda:0"):
                gs.recurrence_bwd(x, x, **dict(dict(grad_h=on(0, B, T, D)), **kw))
        long = on(0, B, 200, D)
        with pytest.raises(TypeError, match="scratch"):
            gs.recurrence_fwd(long, long, scratch=on(bad, 1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gs.recurrence_fwd(x, on(1, B, T, D))
    for call in (lambda: gs.recurrence_fwd(x, x, stream=STREAM), lambda: gs.recurrence_bwd(x, x, x, stream=STREAM)):
        with pytest.raises(ValueError, match="stream belongs to cuda:1"):
            call()


def test_lists_refuse_other_devices():
    import gaussian_splatting_tile_amd as gs
    g = on(0, 8)
    with pytest.raises(TypeError):
        gs.GradList([g, on(1, 8)])
    with pytest.raises(TypeError, match="cuda:0"):
        gs.GradList([g], out=[on(1, 8)])
    with pytest.raises(TypeError):
        gs.Adam([g], [on(1, 8)])
    for call in (gs.grad_norm, lambda grads, **kw: gs.clip_grads(grads, 1.0, **kw)):
        with pytest.raises(ValueError, match="stream belongs to cuda:1"):
            call([g], stream=STREAM)
