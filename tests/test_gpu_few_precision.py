"""What the few-token layer promises about precision, against 64 bits: hidden
activations to more than bf16's precision, relative to each, and one rounding
of y.

Hidden activations.  One expert, W1 = 0 and W2 = 2^20 on the diagonal: y[j] is
2^20 GELU(b1[j]), with one product in each sum, plus the residual, which here
takes away the 64-bit value rounded to y's type, so that y shows what is left.
  bf16 with more than four tokens: two bf16 parts (2^-18 of the value), GELU by
  a polynomial (2^-21) and a density whose exponent, 0.73 x^2 + 1.33, is rounded
  three times (ln 2 * 2^-24 of it each), ten more fp32 roundings;
  otherwise GELU by a polynomial (2^-24) and up to 15 roundings of an fp32 number.
Rounding of y.  Sums of whole numbers, at most 2^24, have no rounding errors of
their own; then y is the 64-bit value rounded once."""
import math

import pytest
import torch

from mixture_experts_layer_11_gb300.decode import FewTokenPass

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def gelu64(x):
    x = x.double()
    return x * 0.5 * torch.special.erfc(-x / math.sqrt(2.0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 3, 5, 16, 64])
@pytest.mark.parametrize("lo,hi", [(-12.0, -3.0), (-3.0, 8.0)])
def test_hidden_activations_hold_their_tails(dtype, T, lo, hi):
    dt, n = TYPES[dtype], 256
    b1 = torch.linspace(lo, hi, n, device=DEV).to(dt)
    W2 = torch.diag(torch.full((n,), 2.0 ** 20, device=DEV)).to(dt)
    exact = 2.0 ** 20 * gelu64(b1)
    near = exact.to(dt)
    fp = FewTokenPass(T, torch.zeros(1, n, dtype=dt, device=DEV), torch.zeros(1, n, n, dtype=dt, device=DEV),
                      b1[None], W2[None], None, 1, 1)
    x = torch.randn(T, n, device=DEV).to(dt)
    y = fp.forward(x, residual=(-near).expand(T, -1).contiguous()).double()
    if dtype == "bf16" and T > 4:
        power = 0.73 * b1.double() ** 2 + 1.33
        rel = 2.0 ** -18 + 2.0 ** -21 + (3 * math.log(2.0) * power + 10) * 2.0 ** -24
    else:
        rel = (1 + 15) * 2.0 ** -24
    # rounding is monotonic: y lies between the rounded ends of what it may have been before
    left = exact - near.double()
    off = rel * exact.abs() + 2.0 ** -24 * near.double().abs() + 1e-37
    low, high = (left - off).to(dt).double(), (left + off).to(dt).double()
    assert ((low <= y) & (y <= high)).all(), float(((y - left).abs() / off).max())
    assert int(fp.status.item()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 4, 6, 40])
def test_y_is_rounded_once(dtype, T):
    # GELU(32) = 32 to all 24 bits and GELU(0) = 0: hidden activations are 32 or 0,
    # W2 whole numbers, so that the sums are exact; a residual that takes most of them away
    dt, d, f = TYPES[dtype], 264, 128
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    whole = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV).to(dt)  # noqa: E731
    b1 = 32 * whole(0, 2, 1, f)
    W2 = whole(0, 129, 1, d, f)
    b2 = whole(0, 200, 1, d)
    sums = W2[0].double() @ b1[0].double() + b2[0].double()
    residual = (whole(-100, 101, T, d).double() - sums.to(dt).double()).to(dt)
    fp = FewTokenPass(T, torch.zeros(1, d, dtype=dt, device=DEV), torch.zeros(1, f, d, dtype=dt, device=DEV),
                      b1, W2, b2, 1, 1)
    y = fp.forward(torch.randn(T, d, device=DEV).to(dt), residual=residual)
    exact = sums + residual.double()
    assert float(sums.max()) < 2 ** 24
    assert torch.equal(y, exact.to(dt))
    y = fp.forward(torch.randn(T, d, device=DEV).to(dt))
    assert torch.equal(y, sums.to(dt).expand(T, -1))
