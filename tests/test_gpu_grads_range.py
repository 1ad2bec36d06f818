"""Clipping where the factor max_norm / norm is below fp32's normal numbers, and
the norm's precision where a thread's sum in fp32 is longest.

Tolerances.  A thread adds the squares of one chunk in fp32: eight 16-byte
vectors, 64 bf16 values, and one value from the chunk's ends, so at most 65
roundings, 65 * 2^-24 of the sum of positive terms, half of it of the norm; the
pair of fp32 numbers over the chunks and the sums in 64 bits add far less, the
norm's own rounding 2^-24: (65 / 2 + 1 + 0.5) * 2^-24.  The factor adds a
rounding, the product two (fp32) and 2^-8 (bf16's 8 bits); a result below 2^-126
is off by up to 2^-149 of itself at each of its two roundings."""
import math

import pytest
import torch

from mixture_experts_layer_11_gb300.grads import GradClip

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
NORM = (65 / 2 + 1.5) * 2.0 ** -24
OUT = {F32: NORM + 3 * 2.0 ** -24, BF16: NORM + 2 * 2.0 ** -24 + 2.0 ** -8}


def norm64(ts):
    big = max(float(t.double().abs().max()) for t in ts)
    return big * math.sqrt(sum(float(((t.double() / big) ** 2).sum()) for t in ts))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("size", [7, 5001, 300001])
@pytest.mark.parametrize("scale,bound", [(1e30, 1e-6), (1e30, 1e-10), (1e33, 1e-3), (1e30, 1e-25),
                                         (1e20, 1e-19), (1e33, 1e-37), (1e10, 1e-30), (1e35, 0.0)])
def test_factors_below_the_normal_numbers(dtype, in_place, size, scale, bound):
    g = torch.Generator(device=DEV)
    g.manual_seed(size)
    t = (torch.randn(size, generator=g, device=DEV) * scale).to(dtype)
    out = None if in_place else torch.full_like(t, 3.0)
    before = t.double()
    want = norm64([t])
    c = GradClip([t], None if in_place else [out])
    assert abs(float(c.clip(bound)) - want) <= NORM * want
    exact = before * (bound / want)
    got = (t if in_place else out).double()
    tiny = 2.0 ** -149 if dtype == F32 else 2.0 ** -133
    assert ((got - exact).abs() <= OUT[dtype] * exact.abs() + 2 * tiny).all()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("power", list(range(-66, -36)) + [38, 39, 40, 41])
def test_norm_where_the_way_of_adding_changes(dtype, power):
    # groups of four around the magnitudes where squares are scaled, alone and beside much smaller ones
    g = torch.Generator(device=DEV)
    g.manual_seed(power + 100)
    t = torch.randn(70001, generator=g, device=DEV) * 2.0 ** power
    small = torch.randn(70001, generator=g, device=DEV) * 2.0 ** (power - 12)
    mixed = torch.where(torch.arange(70001, device=DEV) % 4 == 1, t, small)
    for v in (t.to(dtype), mixed.to(dtype)):
        want = norm64([v])
        assert abs(float(GradClip([v]).norm()) - want) <= NORM * want


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [1.0, 1.0 + 2.0 ** -7, 0.3, 2.0 ** -30])
def test_norm_where_every_rounding_goes_one_way(dtype, value):
    # equal values: the fp32 sums of a thread grow by the same term each time
    for n in (256 * 64, 256 * 64 + 7, 3 * 256 * 64 + 1, 50_000_001):
        t = torch.full((n + 1,), value, dtype=dtype, device=DEV)[1:]
        want = math.sqrt(n) * float(t[0].double())
        assert abs(float(GradClip([t]).norm()) - want) <= NORM * want
