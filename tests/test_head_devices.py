"""``HeadLoss`` launches on its head's device, whichever is current, refuses tensors of
two devices and shapes that do not fit, and tells a device-side error once.  No GPU
needed: the tensors and torch.cuda are stand-ins."""
import pytest
import torch

from mixture_experts_layer_11_gb300 import build as mbuild
from mixture_experts_layer_11_gb300 import ops
from mixture_experts_layer_11_gb300.head import HeadLoss
from test_few_grads_devices import Gpus, Tensor as Plain

I64, F32 = torch.int64, torch.float32


class Tensor(Plain):
    def dim(self):
        return len(self.shape)


@pytest.fixture
def gpus(monkeypatch):
    g = Gpus(monkeypatch)
    for fn in ("moe_head_ce", "moe_head_distill"):
        monkeypatch.setattr(ops, fn, lambda *a, stream: g.calls.append((g.current, stream)))
    monkeypatch.setattr(ops, "moe_head_workspace_size", lambda *a: g.sized.append(g.current) or 64)
    make = lambda *s, dtype=None, device=None: Tensor(  # noqa: E731
        torch.device(device).index, *(s[0] if s and isinstance(s[0], tuple) else s), dtype=dtype or F32)
    for fn in ("empty", "zeros"):
        monkeypatch.setattr(torch, fn, make)
    monkeypatch.setattr(torch, "empty_like", lambda t: make(*t.shape, dtype=t.dtype, device=t.device))
    return g


def tensors(index, t=4, n=3):
    return dict(x=Tensor(index, t, 8), target=Tensor(index, t, dtype=I64), idx=Tensor(index, t, n, dtype=I64),
                logits=Tensor(index, t, n), weight=Tensor(index, t))


@pytest.mark.parametrize("index", [0, 1])
def test_launches_on_its_heads_device(gpus, index):
    head = HeadLoss(4, Tensor(index, 20, 8), entries=3)
    a = tensors(index)
    loss, lse, dx, dW = head.cross_entropy(a["x"], a["target"], weight=a["weight"])
    assert loss is head.loss and dx is head.dx and dW is head.dW and dW.device.index == index
    head.score(a["x"], a["target"])
    head.distill(a["x"], a["idx"], a["logits"])
    assert gpus.calls == [(index, 1000 + index)] * 3 and gpus.sized == [index]
    assert gpus.current == 0


@pytest.mark.parametrize("name", ["x", "target", "idx", "logits", "weight"])
def test_refuses_inputs_on_another_device(gpus, name):
    head = HeadLoss(4, Tensor(0, 20, 8), entries=3)
    a = tensors(0)
    a[name] = tensors(1)[name]
    with pytest.raises(ops.MoEError, match="cuda:1"):
        head.cross_entropy(a["x"], a["target"], weight=a["weight"])
        head.distill(a["x"], a["idx"], a["logits"])
    assert len(gpus.calls) <= 1
    with pytest.raises(ops.MoEError, match="cuda:1"):
        HeadLoss(4, Tensor(0, 20, 8), dW=Tensor(1, 20, 8))


@pytest.mark.parametrize("call", [
    lambda h, a: h.score(Tensor(0, 5, 8), Tensor(0, 5, dtype=I64)),               # more than T tokens
    lambda h, a: h.score(Tensor(0, 4, 16), a["target"]),                          # another width
    lambda h, a: h.score(Tensor(0, 32), a["target"]),
    lambda h, a: h.score(a["x"], Tensor(0, 3, dtype=I64)),
    lambda h, a: h.score(a["x"], Tensor(0, 4, 1, dtype=I64)),
    lambda h, a: h.score(a["x"], Tensor(0, dtype=I64)),
    lambda h, a: h.cross_entropy(a["x"], a["target"], weight=Tensor(0, 3)),
    lambda h, a: h.distill(a["x"], a["idx"], Tensor(0, 4, 2)),
    lambda h, a: h.distill(a["x"], Tensor(0, 4, 4, dtype=I64), Tensor(0, 4, 4)),  # more entries
    lambda h, a: h.distill(a["x"], Tensor(0, 3, 3, dtype=I64), Tensor(0, 3, 3)),
    lambda h, a: h.distill(a["x"], a["target"], a["target"]),
    lambda h, a: h.cross_entropy(a["x"], a["target"], accumulate=True),           # of a bf16 dW
    lambda h, a: HeadLoss(4, h.W, backward=False).cross_entropy(a["x"], a["target"]),
])
def test_refuses_what_does_not_fit(gpus, call):
    head = HeadLoss(4, Tensor(0, 20, 8, dtype=torch.bfloat16), entries=3)
    with pytest.raises(ValueError):
        call(head, tensors(0))
    assert gpus.calls == []


def test_a_head_given_another_shape_or_device_is_refused(gpus):
    head = HeadLoss(4, Tensor(0, 20, 8), entries=3)
    a = tensors(0)
    head.W = Tensor(0, 10, 16)
    with pytest.raises(ValueError, match="W is"):
        head.score(a["x"], a["target"])
    head.W = Tensor(1, 20, 8)
    with pytest.raises(ops.MoEError, match="W on cuda:1"):
        head.score(a["x"], a["target"])
    assert gpus.calls == []


@pytest.mark.parametrize("code", [ops.MOE_ERR_TIMEOUT, ops.MOE_ERR_NONFINITE, ops.MOE_ERR_INVALID])
def test_an_error_is_raised_once(code):
    mbuild.build()
    head = object.__new__(HeadLoss)
    head.status = torch.zeros(1, dtype=torch.int32)
    head.check_status()
    head.status.fill_(code)
    with pytest.raises(ops.MoEError) as e:
        head.check_status()
    assert e.value.code == code
    head.check_status()
