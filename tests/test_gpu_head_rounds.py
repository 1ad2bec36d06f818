"""Scores by objects made with gradients, whose rounds are others than the gradients'."""
import pytest
import torch

from head_util import make, make_entries, near, reference
from mixture_experts_layer_11_gb300 import ops
from mixture_experts_layer_11_gb300.head import HeadLoss

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,d,V", [(4096, 1024, 500), (600, 64, 300), (70001, 8, 40)])
@pytest.mark.parametrize("want_dW", [True, False])
def test_scores_stay_in_an_objects_workspace(T, d, V, dtype, want_dW):
    x, W, target = make(T, d, V, dtype, seed=T)
    target[::7] = -1
    head = HeadLoss(T, W, want_dW=want_dW, piece=256, entries=3)
    # the object's workspace, with a guard behind it
    n = head.ws.numel()
    assert n >= ops.moe_head_workspace_size(ops.make_head(T, V, d, dtype, 3, 256))
    big = torch.full((n + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    head.ws = big[:n]
    head._owned = (head.ws.data_ptr(), head._owned[1])
    alone = [v.clone() for v in HeadLoss(T, W, backward=False).score(x, target)]
    want, bound = reference(x, W, target, mean=True)
    first = None
    for _ in range(2):
        grads = head.cross_entropy(x, target, mean=True)
        near("dx", grads[2], want["dx"], bound["dx"])
        first = first or [v.clone() for v in grads if v is not None]
        assert all(torch.equal(a, b) for a, b in zip(first, (v for v in grads if v is not None)))
        got = head.score(x, target)
        assert all(torch.equal(a, b) for a, b in zip(alone, got))
        for t in (1, 60, 129, T // 2):
            loss, _ = head.score(x[:t], target[:t])
            near("loss", loss, want["loss"][:t], bound["loss"][:t])
    idx, logits = make_entries(T, 3, V, target.clamp(min=0), distinct=False)
    head.distill(x, idx, logits)
    torch.cuda.synchronize()
    assert bool((big[n:] == 0xA5).all())
    head.check_status()
