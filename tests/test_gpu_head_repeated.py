"""Indices that a teacher's list holds more than once: one entry's value of the gradient
by the logits, the sum of all in the list's order, whichever lane comes last."""
import pytest
import torch

from head_util import make, make_entries, near, reference
from mixture_experts_layer_11_gb300.head import HeadLoss

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [64, 300])
def test_the_order_of_the_first_two_does_not_count(T, dtype):
    # (a + b) + c has the bits of (b + a) + c, and not those of (c + b) + a.  The softmax's
    # own sum adds lanes 16 apart first, then those 8 apart: entries 0, 16 and 24 keep its
    # bits, and with them q's, when the first two change places
    V = 129
    x, W, target = make(T, 64, V, dtype, seed=T)
    idx = torch.full((T, 25), -1, device="cuda")
    idx[:, [0, 16, 24]] = target[:, None]
    logits = 3.0 * torch.randn(T, 25, device="cuda")
    a, b, c = torch.softmax(logits[:, [0, 16, 24]], 1).unbind(1)
    assert ((a + b) + c != (c + b) + a).any()
    swapped = logits.clone()
    swapped[:, 0], swapped[:, 16] = logits[:, 16], logits[:, 0]
    head = HeadLoss(T, W, dW=torch.empty(V, 64, device="cuda"), entries=25)
    one = [v.clone() for v in head.distill(x, idx, logits)[2:]]
    two = head.distill(x, idx, swapped)[2:]
    assert all(torch.equal(u, v) for u, v in zip(one, two))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K", [3, 33, 128])
def test_repeated_entries_have_the_same_bits_every_time(K, dtype):
    # few indices, many times each, some across the borders of 128 and 2048 entries
    T, V = 200, 5000
    x, W, target = make(T, 64, V, dtype, seed=K)
    _, logits = make_entries(T, K, V, target, seed=K)
    few = torch.tensor([0, 127, 128, 2047, 2048, 4999], device="cuda")
    idx = few[torch.randint(0, 6, (T, K), device="cuda")]
    idx[::5, ::3] = -1
    idx[7] = 2048
    head = HeadLoss(T, W, entries=K)
    want, bound = reference(x, W, idx=idx, logits=logits, temperature=1.5)
    a = None
    for _ in range(4):
        head.ws.random_(0, 256)
        got = head.distill(x, idx, logits, temperature=1.5)
        for k, v in zip(("loss", "lse", "dx"), got):
            near(k, v, want[k], bound[k])
        near("dW", got[3], want["dW"], bound["dW32" if dtype == F32 else "dW"])
        a = a or [v.clone() for v in got]
        assert all(torch.equal(u, v) for u, v in zip(a, got))
    head.check_status()
