"""dW in fp32 over many rows, where nothing but the sum itself is rounded: with W = 0 every
probability is 1/256 and G is 1/256 or -255/256, exact in bf16, and so is x.  The tensor
cores add 16 products a step to the accumulator and drop what is below its last bit: a
chain of n products is off by at most n / 16 steps of 2^-22 (the accumulator's last bit,
2^-23 of it, and as much for the products' own alignment) of the sum of magnitudes, and
always towards zero.  A chain is a round's rows, 65536 at most; rounds are added in fp32."""
import pytest
import torch

from head_util import D
from mixture_experts_layer_11_gb300.head import HeadLoss

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,piece", [(65536, 0), (65536, 8192), (4096, 0)])
def test_fp32_dW_over_many_rows(T, piece):
    # 80 column tiles: most of them whole, whose sums are not cut into parts
    V, d = 256, 80 * 256
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.rand(T, d, generator=g, device="cuda").bfloat16()
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    W = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    head = HeadLoss(T, W, dW=torch.empty(V, d, device="cuda"), want_dx=False, piece=piece)
    got = head.cross_entropy(x, target)[3].to(D)
    head.check_status()
    want, size = torch.zeros(V, d, dtype=D, device="cuda"), torch.zeros(V, d, dtype=D, device="cuda")
    for a in range(0, T, 4096):
        G = torch.full((min(4096, T - a), V), 1 / 256, dtype=D, device="cuda")
        G[torch.arange(len(G)), target[a:a + 4096]] -= 1.0
        part = x[a:a + 4096].to(D)
        want += G.T @ part
        size += G.abs().T @ part
    off = (got - want) / size
    steps = min(T, piece or T) / 16
    print(f"T {T} piece {piece}: off {float(off.abs().max()):.2e} of the magnitudes, norm "
          f"{float((got - want).norm() / want.norm()):.2e}, norm over magnitudes' {float((got - want).norm() / size.norm()):.2e}")
    assert float(off.abs().max()) <= steps * 2.0 ** -22 + (T / (piece or T)) * 2.0 ** -24
