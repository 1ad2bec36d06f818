"""``HeadLoss`` of which neither gradient is wanted makes the calls that scores make: no
workspace for probabilities, none written.  Without a GPU on stand-ins."""
import pytest
import torch

from mixture_experts_layer_11_gb300 import ops
from mixture_experts_layer_11_gb300.head import HeadLoss
from test_head_devices import Tensor, gpus, tensors  # noqa: F401


def test_neither_gradient_is_scores(gpus, monkeypatch):  # noqa: F811
    grads = []
    monkeypatch.setattr(ops, "moe_head_workspace_size", lambda h, g=None: grads.append(g) or 64)
    for fn, at in (("moe_head_ce", 6), ("moe_head_distill", 8)):
        monkeypatch.setattr(ops, fn, lambda *a, stream, at=at: grads.append(a[at]))
    head = HeadLoss(4, Tensor(0, 20, 8), entries=3, want_dx=False, want_dW=False)
    a = tensors(0)
    for got in (head.cross_entropy(a["x"], a["target"], weight=a["weight"], mean=True),
                head.distill(a["x"], a["idx"], a["logits"], scale=2.0), (*head.score(a["x"], a["target"]), None, None)):
        assert got[0] is head.loss and got[1] is head.lse and got[2:] == (None, None)
    assert grads == [None] * 4
    # what is refused stays refused
    with pytest.raises(ValueError):
        head.cross_entropy(a["x"], a["target"], weight=Tensor(0, 3))
    with pytest.raises(ops.MoEError):
        head.cross_entropy(a["x"], a["target"], weight=Tensor(0, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        HeadLoss(4, Tensor(0, 20, 8), backward=False).cross_entropy(a["x"], a["target"])
    grads.clear()
    HeadLoss(4, Tensor(0, 20, 8), want_dx=False).cross_entropy(a["x"], a["target"])
    assert len(grads) == 2 and all(g is not None for g in grads)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [40, 300])
def test_neither_gradient_on_a_gpu(T, dtype):
    from head_util import make, make_entries
    x, W, target = make(T, 64, 700, dtype)
    target[::5] = -1
    idx, logits = make_entries(T, 6, 700, target.clamp(min=0))
    neither, scores = (HeadLoss(T, W, entries=6, **k) for k in (dict(want_dx=False, want_dW=False), dict(backward=False)))
    assert neither.ws.numel() == scores.ws.numel()
    want = [v.clone() for v in scores.score(x, target)]
    got = neither.cross_entropy(x, target, weight=torch.rand(T, device="cuda"), mean=True)
    assert got[2:] == (None, None) and all(torch.equal(a, b) for a, b in zip(want, got))
    want = [v.clone() for v in scores.distill(x, idx, logits)[:2]]
    got = neither.distill(x, idx, logits)
    assert got[2:] == (None, None) and all(torch.equal(a, b) for a, b in zip(want, got))
    neither.check_status()
