"""The global gradient norm and clipping against the formulas in 64 bits.

Tolerances: a thread sums at most 48 squares in fp32 before it goes on in 64
bits (48 * 2^-24 of the sum, half of it of the norm), and the norm is rounded
once: 32 * 2^-24.  The factor adds one rounding and the product one more (2^-8
in bf16)."""
import math

import pytest
import torch

from mixture_experts_layer_11_gb300 import ops
from mixture_experts_layer_11_gb300.grads import GradClip

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
NORM = 32 * 2.0 ** -24
OUT = {F32: NORM + 3 * 2.0 ** -24, BF16: NORM + 2.0 ** -8}


def exact(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


def make(sizes, dtypes=(F32,), scale=1.0, seed=0, shift=0):
    """Gradients as views of one buffer per type, `shift` elements from its start."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out, at = [], {}
    kinds = [dtypes[i % len(dtypes)] for i in range(len(sizes))]
    flat = {dt: torch.randn(shift + sum(n for n, q in zip(sizes, kinds) if q == dt), generator=g,
                            device=DEV).mul_(scale).to(dt) for dt in dtypes}
    for n, dt in zip(sizes, kinds):
        a = at.get(dt, shift)
        out.append(flat[dt][a:a + n])
        at[dt] = a + n
    return out


def check(ts, bound, outs=None):
    before = [t.clone() for t in ts]
    want = exact(before)
    c = GradClip(ts, outs)
    got = c.clip(bound)
    assert abs(float(got) - want) <= NORM * want
    factor = bound / want if want > bound else 1.0
    for t, b, o in zip(ts, before, outs or ts):
        if factor == 1.0:
            assert torch.equal(o, b)
        else:
            assert ((o.double() - b.double() * factor).abs() <= OUT[b.dtype] * b.double().abs() * factor + 1e-45).all()
        if outs is not None:
            assert torch.equal(t, b)
    assert int(c.status.item()) == 0
    return c


SIZES = [[1], [3], [8], [4096], [16383], [16384], [16385], [100003], [1, 1, 1], [5, 0, 7, 0],
         [16384, 16384], [3, 70001, 2, 9, 33000], [65536 * 20 + 1], list(range(1, 301)),
         [0, 0, 5], [7] * 1000]


@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (F32, BF16)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip(sizes, dtypes):
    for shift in (0, 1, 3):
        ts = make(sizes, dtypes, shift=shift, seed=shift)
        n = GradClip(ts).norm()
        assert abs(float(n) - exact(ts)) <= NORM * exact(ts)
        check(ts, 0.25 * exact(ts))
        check(ts, 4.0 * exact(ts))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("a,b", [(0, 0), (0, 1), (3, 5), (7, 2), (4, 8), (1, 1)])
def test_into_other_buffers(dtype, a, b):
    # any alignment of the two sides against each other
    sizes = [100001, 3, 20000, 1]
    ts = make(sizes, (dtype,), shift=a)
    outs = [o.fill_(9) for o in make(sizes, (dtype,), shift=b, seed=1)]
    check(ts, 0.5 * exact(ts), outs)
    check(ts, 2.0 * exact(ts), outs)


def test_nothing_outside_is_written():
    for dt in (F32, BF16):
        buf = torch.full((50000,), 3.0, dtype=dt, device=DEV)
        GradClip([buf[5:20001], buf[30003:30004], buf[40000:49999]]).clip(1.0)
        for s in (slice(0, 5), slice(20001, 30003), slice(30004, 40000), slice(49999, None)):
            assert (buf[s] == 3).all()
        assert (buf[5:20001] != 3).all()


@pytest.mark.parametrize("scale", [1e-42, 1e-38, 1e-30, 1e-20, 1e-12, 1e-6, 1e6, 1e15, 1e20, 1e30, 1e34])
def test_the_whole_range(scale):
    ts = [t.float() * scale for t in make([40000, 17])]
    check(ts, 0.5 * exact(ts))


def test_mixed_magnitudes():
    ts = [torch.tensor([1e30, 1e-30, 0.0, 1.0] * 99, device=DEV), torch.full((999,), 1e-25, device=DEV)]
    check(ts, 1.0)
    ts = [torch.tensor([1e-25, 0.0, 1e-44, 1e-20] * 50, device=DEV), torch.full((3,), 1e-38, device=DEV)]
    check(ts, 1e-22)


def test_all_zero_and_empty():
    z = torch.zeros(1000, device=DEV)
    assert float(check([z], 0.0).total) == 0.0
    for ts in ([], [z[:0]], [z[:0], z[:0]]):
        c = GradClip(ts)
        c.total.fill_(5)
        assert float(c.norm()) == 0.0
        c.total.fill_(5)
        assert float(c.clip(1.0)) == 0.0
        assert int(c.status.item()) == 0


def test_a_first_launch_without_elements():
    ts = [torch.zeros(0, device=DEV)] * 1000 + make([5, 3])
    c = GradClip(ts)
    want = exact(ts)
    assert abs(float(c.clip(0.5 * want)) - want) <= NORM * want
    assert abs(exact(ts) - 0.5 * want) <= 2 * NORM * want


def test_bounds():
    ts = make([5000, 77], (F32, BF16))
    norm = float(GradClip(ts).norm())
    before = [t.clone() for t in ts]
    GradClip(ts).clip(math.inf)
    assert all(torch.equal(t, b) for t, b in zip(ts, before))
    GradClip(ts).clip(norm)          # at the bound: not over it
    assert all(torch.equal(t, b) for t, b in zip(ts, before))
    GradClip(ts).clip(0.0)
    assert all((t == 0).all() for t in ts)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 20000, 33332])
def test_not_finite(bad, at):
    for dt in (F32, BF16):
        ts = make([33333, 10], (dt,))
        ts[0][at] = bad
        before = [t.clone() for t in ts]
        outs = [torch.zeros_like(t) for t in ts]
        c = GradClip(ts, outs)
        n = float(c.clip(1e-3))
        assert math.isnan(n) if math.isnan(bad) else n == math.inf
        assert int(c.status.item()) == ops.MOE_ERR_NONFINITE
        for t, o, b in zip(ts, outs, before):
            assert torch.equal(t.nan_to_num(5.0), b.nan_to_num(5.0))
            assert torch.equal(o.nan_to_num(5.0), b.nan_to_num(5.0))
        c = GradClip(ts)
        c.norm()
        assert int(c.status.item()) == ops.MOE_ERR_NONFINITE


def test_a_nan_beside_any_magnitude_is_seen():
    for v in (1e-30, 1.0, 1e30, 0.0):
        t = torch.full((64,), v, device=DEV)
        t[9] = math.nan
        assert math.isnan(float(GradClip([t]).norm()))


def test_same_bits_every_time_on_any_stream():
    ts = make([300001, 5, 12345], (F32, BF16))
    outs = [torch.empty_like(t) for t in ts]
    c = GradClip(ts, outs)
    n = c.clip(1.0).clone()
    want = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for fill in (0, 0xFF):
            c.ws.fill_(fill)
            [o.zero_() for o in outs]
            m = c.clip(1.0).clone()
    side.synchronize()
    assert torch.equal(n, m) and all(torch.equal(a, b) for a, b in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.clip(1.0)
    for t in ts:
        t.mul_(3)
    g.replay()
    assert abs(float(c.total) - 3 * float(n)) <= 2e-2 * float(n)


def test_right_behind_the_kernels_that_make_the_gradients():
    # the launches overlap the end of the kernel before them, not its results
    src = [torch.randn(300001, device=DEV) * (i + 1) for i in range(20)]
    t = torch.empty(300001, device=DEV)
    c = GradClip([t])
    norms = []
    for s in src:
        t.copy_(s)
        norms.append(c.clip(1.0).clone())
        norms.append(c.norm().clone())
    for s, a, b in zip(src, norms[::2], norms[1::2]):
        assert abs(float(a) - exact([s])) <= NORM * exact([s])
        assert abs(float(b) - 1.0) <= 3 * NORM


def test_beyond_32_bits():
    n = 2 ** 31 + 5
    t = torch.full((n,), 0.5, dtype=BF16, device=DEV)
    t[-1] = 3.0
    norm = math.sqrt((n - 1) * 0.25 + 9.0)
    c = GradClip([t[1:], t[:1]])
    assert abs(float(c.clip(norm / 4)) - norm) <= NORM * norm
    assert float(t[0]) == float(t[-2]) == 0.125 and float(t[-1]) == 0.75
    assert float(t.min()) == 0.125


def test_refusals():
    t = torch.zeros(8, 8, device=DEV)
    with pytest.raises(ops.MoEError):
        GradClip([t.t()[:, :3]])
    with pytest.raises(ops.MoEError):
        GradClip([t.double()])
    with pytest.raises(ops.MoEError):
        GradClip([t], [t.to(BF16)])
    with pytest.raises(ops.MoEError):
        GradClip([t], [t[:4]])
    with pytest.raises(ops.MoEError):
        GradClip([t]).clip(-1.0)
