"""The classes around the few-token layer and the gradient norm launch on their
tensors' device, whichever is current, and refuse tensors of two devices.  No
GPU needed: the tensors and torch.cuda are stand-ins."""
import contextlib

import pytest
import torch

from mixture_experts_layer_11_gb300 import ops
from mixture_experts_layer_11_gb300.decode import FewTokenPass
from mixture_experts_layer_11_gb300.grads import GradClip


class Tensor:
    """What the classes ask of a tensor, on device `index`."""
    is_cuda = True

    def __init__(self, index, *shape, dtype=torch.float32):
        self.device, self.shape, self.dtype = torch.device("cuda", index), torch.Size(shape), dtype

    def get_device(self):
        return self.device.index

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def __getitem__(self, i):
        return Tensor(self.device.index, i.stop, *self.shape[1:])


def weights(index, other=None, name=None):
    shapes = dict(Wg=(2, 8), W1=(2, 16, 8), b1=(2, 16), W2=(2, 8, 16), b2=(2, 8), beta=(2,))
    return {n: Tensor(other if n == name else index, *s) for n, s in shapes.items()}


class Gpus:
    """torch.cuda with two devices: what is current, and at which device and on
    which stream the library was called."""

    def __init__(self, monkeypatch):
        self.current, self.calls, self.sized = 0, [], []
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "device", self.device)
        monkeypatch.setattr(ops, "raw_stream", lambda index: 1000 + index)
        for fn in ("moe_layer_few", "moe_grad_norm", "moe_grad_clip"):
            monkeypatch.setattr(ops, fn, lambda *a, stream: self.calls.append((self.current, stream)))
        for fn in ("moe_layer_few_workspace_size", "moe_grad_workspace_size"):
            monkeypatch.setattr(ops, fn, lambda *a: self.sized.append(self.current) or 64)
        for fn in ("empty", "zeros"):
            monkeypatch.setattr(torch, fn, lambda *s, dtype=None, device=None: Tensor(
                torch.device(device).index, *(s[0] if s and isinstance(s[0], tuple) else s), dtype=dtype))

    @contextlib.contextmanager
    def device(self, dev):
        was, self.current = self.current, dev if isinstance(dev, int) else dev.index
        try:
            yield
        finally:
            self.current = was


@pytest.fixture
def gpus(monkeypatch):
    return Gpus(monkeypatch)


def few(p):
    return FewTokenPass(4, p["Wg"], p["W1"], p["b1"], p["W2"], p["b2"], 1, 1, beta=p["beta"])


@pytest.mark.parametrize("index", [0, 1])
def test_few_launches_on_its_weights_device(gpus, index):
    fp = few(weights(index))
    x = Tensor(index, 4, 8)
    assert fp.forward(x, x) is fp.y and fp.y.device.index == index
    assert gpus.calls == [(index, 1000 + index)] and gpus.sized == [index]
    assert gpus.current == 0


@pytest.mark.parametrize("index", [0, 1])
def test_clip_launches_on_its_gradients_device(gpus, index):
    clip = GradClip([Tensor(index, 5), Tensor(index, 7, dtype=torch.bfloat16)])
    assert clip.norm() is clip.total and clip.clip(1.0) is clip.total
    assert gpus.calls == [(index, 1000 + index)] * 2 and gpus.sized == [index]
    assert gpus.current == 0 and clip.total.device.index == index


@pytest.mark.parametrize("name", ["Wg", "W1", "b1", "W2", "b2", "beta"])
def test_few_refuses_weights_on_two_devices(gpus, name):
    with pytest.raises(ops.MoEError, match="cuda:0.*cuda:1|cuda:1.*cuda:0"):
        few(weights(0, 1, name))


def test_few_refuses_inputs_on_another_device(gpus):
    fp = few(weights(0))
    here, there = Tensor(0, 4, 8), Tensor(1, 4, 8)
    for x, residual, out in ((there, None, None), (here, there, None), (here, None, there)):
        with pytest.raises(ops.MoEError, match="cuda:1"):
            fp.forward(x, residual, out=out)
    assert gpus.calls == []


def test_clip_refuses_tensors_on_two_devices(gpus):
    a, b = Tensor(0, 5), Tensor(1, 5)
    with pytest.raises(ops.MoEError, match="cuda:1"):
        GradClip([a, b])
    with pytest.raises(ops.MoEError, match="cuda:1"):
        GradClip([a, a], [a, b])
