"""Losses over a vocabulary head and their gradients against the formulas in 64
bits; the bounds are derived in ``head_util``."""
import pytest
import torch

from head_util import D, make, make_entries, near, reference
from mixture_experts_layer_11_gb300 import ops
from mixture_experts_layer_11_gb300.head import HeadLoss

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = [F32, BF16]


def check(head, x, target=None, idx=None, logits=None, temperature=1.0, weight=None, scale=1.0,
          mean=False):
    want, bound = reference(x, head.W, target, idx, logits, temperature, weight, scale, mean)
    if target is not None:
        got = head.cross_entropy(x, target, weight=weight, scale=scale, mean=mean)
    else:
        got = head.distill(x, idx, logits, temperature=temperature, weight=weight, scale=scale, mean=mean)
    torch.cuda.synchronize()
    near("loss", got[0], want["loss"], bound["loss"])
    near("lse", got[1], want["lse"], bound["lse"])
    if got[2] is not None:
        near("dx", got[2], want["dx"], bound["dx"])
    if got[3] is not None:
        near("dW", got[3], want["dW"], bound["dW32" if got[3].dtype == F32 else "dW"])
    return got


SIZES = [(1, 8, 1), (1, 64, 5), (3, 72, 127), (2, 16, 128), (33, 64, 129), (64, 520, 1000), (127, 64, 257),
         (128, 136, 511), (129, 64, 513), (255, 32, 777), (256, 64, 1000), (257, 264, 300), (600, 128, 2049)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,V", SIZES)
def test_cross_entropy(T, d, V, dtype):
    x, W, target = make(T, d, V, dtype, seed=T + V)
    head = HeadLoss(T, W)
    check(head, x, target)
    check(head, x, target, scale=0.37, mean=True)
    head.check_status()


@pytest.mark.parametrize("kind", ["ce", "distill"])
@pytest.mark.parametrize("T,d,V", [(4100, 2056, 10007), (4096, 1024, 20000), (5000, 520, 30001)])
def test_long_calls(T, d, V, kind):
    # whole waves of tiles and cut ones behind them; the two gradients in a launch each
    x, W, target = make(T, d, V, BF16, seed=d)
    head = HeadLoss(T, W, entries=5)
    if kind == "ce":
        target[::9] = -1
        check(head, x, target, mean=True)
    else:
        idx, logits = make_entries(T, 5, V, target, distinct=False)
        check(head, x, idx=idx, logits=logits, temperature=1.5, weight=torch.rand(T, device="cuda"), mean=True)
    head.check_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,V", SIZES + [(200, 64, 40000)])
def test_score(T, d, V, dtype):
    x, W, target = make(T, d, V, dtype, seed=T * V)
    target[::3] = -1
    head = HeadLoss(T, W, backward=False)
    want, bound = reference(x, W, target)
    loss, lse = head.score(x, target)
    near("loss", loss, want["loss"], bound["loss"])
    near("lse", lse, want["lse"], bound["lse"])
    head.check_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [1, 2, 31, 32, 33, 128])
@pytest.mark.parametrize("T,d,V", [(1, 64, 300), (65, 72, 1001), (257, 64, 515)])
def test_distill(T, d, V, K, dtype):
    x, W, target = make(T, d, V, dtype, seed=K)
    idx, logits = make_entries(T, K, V, target, seed=K)
    head = HeadLoss(T, W, entries=K)
    check(head, x, idx=idx, logits=logits)
    check(head, x, idx=idx, logits=logits, temperature=2.5, scale=3.0, mean=True)
    check(head, x, idx=idx, logits=logits, temperature=0.5)
    head.check_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [1, 5, 128])
@pytest.mark.parametrize("T,d,V", [(1, 64, 300), (8, 72, 33), (40, 64, 5000), (64, 264, 1001), (65, 64, 1001),
                                   (128, 64, 40000), (129, 64, 700), (300, 72, 1025)])
def test_distill_without_gradients(T, d, V, K, dtype):
    # up to 64 (fp32) or 128 rows take tiles of other widths, in which rows are tokens
    x, W, target = make(T, d, V, dtype, seed=K + T)
    idx, logits = make_entries(T, K, V, target, seed=K, distinct=False)
    if T > 3:
        idx[1] = -1                                     # nothing left
        x[1] = float("nan")
        idx[2, 0] = -1
        logits[3, K // 2:] = float("-inf")
    head = HeadLoss(T, W, entries=K, backward=False)
    for tau in (1.0, 3.0):
        want, bound = reference(x, W, idx=idx, logits=logits, temperature=tau)
        loss, lse, dx, dW = head.distill(x, idx, logits, temperature=tau)
        assert dx is None and dW is None
        near("loss", loss, want["loss"], bound["loss"])
        near("lse", lse, want["lse"], bound["lse"])
    head.check_status()


@pytest.mark.parametrize("dtype", DTYPES)
def test_entries_absent_and_repeated(dtype):
    T, d, V, K = 150, 64, 700, 24
    x, W, target = make(T, d, V, dtype)
    idx, logits = make_entries(T, K, V, target)
    idx[:50, 5:9] = idx[:50, 4:5]                       # an index five times
    idx[10:20] = idx[10:20, :1]                         # a list of one index
    idx[20:40, 7:] = -1                                 # short lists
    idx[40:45, :3] = -7                                 # absent in front
    logits[45:50, ::2] = float("-inf")                  # masked by the logit
    logits[50:55, 1::2] = torch.finfo(F32).min          # ... by the type's lowest value
    logits[55:57] = torch.finfo(F32).min                # everywhere: an even distribution
    idx[60:63] = -1                                     # nothing left
    logits[63:66] = float("-inf")
    logits[66:70, 3] = float("nan")                     # a NaN where the entry is absent
    idx[66:70, 3] = -1
    x[60:66] = float("nan")                             # rows that are ignored hold anything
    head = HeadLoss(T, W, entries=K)
    for tau in (1.0, 0.25):
        got = check(head, x, idx=idx, logits=logits, temperature=tau, mean=True)
    assert not got[2][60:66].float().any() and not got[0][60:66].any()
    head.check_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pattern", ["first", "last", "odd", "one", "all"])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_ignored_tokens(T, pattern, dtype):
    x, W, target = make(T, 64, 333, dtype, seed=T)
    t = torch.arange(T, device="cuda")
    drop = {"first": t < T // 2, "last": t >= T // 2, "odd": t % 2 == 1, "one": t != T // 3,
            "all": t >= 0}[pattern]
    target[drop] = -100
    x[drop] = float("nan")
    x[drop, ::2] = float("inf")
    head = HeadLoss(T, W)
    got = check(head, x, target, mean=True)
    assert not got[0][drop].any() and not got[1][drop].any() and not got[2][drop].float().any()
    scores = HeadLoss(T, W, backward=False)
    loss, lse = scores.score(x, target)
    assert not loss[drop].any() and not lse[drop].any() and torch.isfinite(loss).all()
    head.check_status()
    scores.check_status()


@pytest.mark.parametrize("dtype", DTYPES)
def test_weights(dtype):
    T = 301
    x, W, target = make(T, 64, 450, dtype)
    target[5::7] = -1
    weight = torch.randn(T, device="cuda")
    weight[::4] = 0.0
    weight[5] = float("nan")                            # of an ignored token
    want, _ = reference(x, W, target)
    w = torch.where(target >= 0, weight, 0.0)
    head = HeadLoss(T, W)
    want, bound = reference(x, W, target, weight=w, scale=0.1, mean=True)
    got = head.cross_entropy(x, target, weight=weight, scale=0.1, mean=True)
    for k, v in zip(("loss", "lse", "dx", "dW"), got):
        near(k, v, want[k], bound["dW32" if k == "dW" and dtype == F32 else k])


@pytest.mark.parametrize("dtype", DTYPES)
def test_sure_and_surprised(dtype):
    # targets that are nearly certain (p - 1 has few of p's bits) and ones that are far off
    T, d, V = 128, 64, 900
    x, W, target = make(T, d, V, dtype, spread=0.5, boost=0.0)
    best = W[target].float()
    lift = torch.linspace(-150, 150, T, device="cuda")[:, None]
    x = (x.float() + lift * best / best.square().sum(1, keepdim=True)).to(dtype)
    head = HeadLoss(T, W)
    check(head, x, target)
    # logits whose largest lies far above the target's, in another block and in the same
    other = (target + 1) % V
    check(head, x, other)
    head.check_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,piece", [(600, 256), (513, 200), (1030, 512), (300, 256)])
def test_pieces(T, piece, dtype):
    x, W, target = make(T, 72, 400, dtype, seed=piece)
    target[::5] = -1
    whole, cut = HeadLoss(T, W), HeadLoss(T, W, piece=piece)
    check(cut, x, target, mean=True)
    a = [v.clone() for v in whole.cross_entropy(x, target)]
    b = cut.cross_entropy(x, target)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    target[256:] = -1                                   # pieces without any row
    check(cut, x, target, mean=True)
    target[:] = -1
    got = check(cut, x, target, mean=True)
    assert not got[3].float().any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("piece", [0, 256])
def test_accumulate(dtype, piece):
    T, d, V = 290, 64, 333
    x, W, target = make(T, d, V, dtype)
    dW = torch.randn(V, d, device="cuda")
    before = dW.clone()
    head = HeadLoss(T, W, dW=dW, piece=piece)
    want, bound = reference(x, W, target)
    for i in range(2):
        head.cross_entropy(x, target, accumulate=True)
    off = (dW.double() - before.double() - 2 * want["dW"]).abs()
    # two additions (a piece more each): half a step of what is in the buffer each
    assert (off <= 2 * bound["dW32"] + 6 * 2.0 ** -24 * (before.abs() + 2 * want["dW"].abs() + 1)).all()
    head.cross_entropy(x, target)
    near("dW", dW, want["dW"], bound["dW32"])
    target[:] = -1
    kept = dW.clone()
    head.cross_entropy(x, target, accumulate=True)
    assert torch.equal(dW, kept)
    head.cross_entropy(x, target)
    assert not dW.any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_gradient_only(dtype):
    T, d, V = 70, 64, 333
    x, W, target = make(T, d, V, dtype)
    both = [v.clone() for v in HeadLoss(T, W).cross_entropy(x, target)]
    a = HeadLoss(T, W, want_dW=False).cross_entropy(x, target)
    b = HeadLoss(T, W, want_dx=False).cross_entropy(x, target)
    assert a[3] is None and b[2] is None
    assert torch.equal(a[2], both[2]) and torch.equal(b[3], both[3])


@pytest.mark.parametrize("dtype", DTYPES)
def test_fewer_tokens_than_made_for(dtype):
    x, W, target = make(700, 64, 500, dtype)
    idx, logits = make_entries(700, 9, 500, target)
    head = HeadLoss(700, W, entries=16, piece=512)
    guard = head.dx.clone()
    for t in (0, 1, 128, 129, 512, 513, 700):
        head.dx.fill_(7.0)
        check(head, x[:t], target[:t], mean=True)
        assert (head.dx[t:] == 7.0).all()               # rows behind the last are left alone
        check(head, x[:t], idx=idx[:t], logits=logits[:t], temperature=1.5)
    del guard
    head.check_status()


def test_bad_indices_are_reported():
    for dtype in DTYPES:
        x, W, target = make(40, 64, 100, dtype)
        idx, logits = make_entries(40, 4, 100, target)
        target[3], target[7] = 100, 1 << 40
        for backward in (False, True):
            head = HeadLoss(40, W, backward=backward, entries=4)
            if backward:
                check(head, x, target)                  # as if they had no target
            else:
                loss, _ = head.score(x, target)
                assert loss[3] == 0 and loss[7] == 0
            with pytest.raises(ops.MoEError) as e:
                head.check_status()
            assert e.value.code == ops.MOE_ERR_INVALID
            head.check_status()                         # told once
        idx[5, 2] = 100
        check(head, x, idx=idx, logits=logits)
        with pytest.raises(ops.MoEError):
            head.check_status()


def test_nonfinite_losses_are_reported():
    for dtype in DTYPES:
        for bad in (float("nan"), float("inf")):
            x, W, target = make(300, 64, 100, dtype)
            x[200, 3] = bad
            head = HeadLoss(300, W)
            loss, lse, dx, _ = head.cross_entropy(x, target)
            assert not torch.isfinite(loss[200]) or not torch.isfinite(lse[200])
            others = torch.arange(300, device="cuda") != 200
            want, bound = reference(x[others], W, target[others])
            near("loss", loss[others], want["loss"], bound["loss"])
            near("dx", dx[others], want["dx"], bound["dx"])
            with pytest.raises(ops.MoEError) as e:
                head.check_status()
            assert e.value.code == ops.MOE_ERR_NONFINITE


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradients_against_differences(dtype):
    # the loss's own values along a direction, central differences in 64 bits of the
    # formula, against the gradients that the kernels return
    T, d, V, K = 20, 32, 90, 6
    x, W, target = make(T, d, V, dtype)
    idx, logits = make_entries(T, K, V, target)
    weight = torch.rand(T, device="cuda")
    head = HeadLoss(T, W, entries=K)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for kind in ("ce", "distill"):
        args = dict(target=target) if kind == "ce" else dict(idx=idx, logits=logits, temperature=2.0)
        if kind == "ce":
            _, _, dx, dW = head.cross_entropy(x, target, weight=weight, mean=True)
        else:
            _, _, dx, dW = head.distill(x, idx, logits, temperature=2.0, weight=weight, mean=True)
        _, bound = reference(x, W, weight=weight, mean=True, **args)
        total = lambda a, b: float((weight.to(D) * reference(a, b, **args)[0]["loss"]).sum()) / T  # noqa: E731
        x64, W64, step = x.to(D), W.to(D), 1e-5
        ux = torch.randn(x.shape, generator=g, device="cuda", dtype=D)
        uW = torch.randn(W.shape, generator=g, device="cuda", dtype=D)
        for got, u, e, f in ((dx, ux, bound["dx"], lambda s: total(x64 + s * ux, W64)),
                             (dW, uW, bound["dW"], lambda s: total(x64, W64 + s * uW))):
            slope = (f(step) - f(-step)) / (2 * step)
            assert abs(float((got.to(D) * u).sum()) - slope) <= float((e * u.abs()).sum()) + 1e-6


@pytest.mark.parametrize("dtype", DTYPES)
def test_same_bits_every_time(dtype):
    x, W, target = make(500, 264, 3001, dtype)
    head = HeadLoss(500, W)
    a = [v.clone() for v in head.cross_entropy(x, target)]
    for _ in range(3):
        head.ws.random_(0, 256)                         # nothing is kept in the workspace
        b = head.cross_entropy(x, target)
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_another_stream_and_a_graph():
    x, W, target = make(300, 64, 700, BF16)
    idx, logits = make_entries(300, 8, 700, target)
    want = [v.clone() for v in HeadLoss(300, W).cross_entropy(x, target)]
    soft = [v.clone() for v in HeadLoss(300, W, entries=8).distill(x, idx, logits)]
    a, b = HeadLoss(300, W), HeadLoss(300, W, entries=8)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = a.cross_entropy(x, target)
    stream.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        got = a.cross_entropy(x, target)
    with torch.cuda.graph(g2):
        got2 = b.distill(x, idx, logits)
    keep = [x.clone(), target.clone()]
    for _ in range(2):
        x.copy_(keep[0])
        target.copy_(keep[1])
        for t in (*got, *got2):
            t.fill_(float("nan"))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, got))
        assert all(torch.equal(u, v) for u, v in zip(soft, got2))
        x.mul_(0.5)                                     # other inputs, other tokens ignored
        target[::2] = -1
        g1.replay()
        w, e = reference(x, W, target)
        near("dx", got[2], w["dx"], e["dx"])
        near("dW", got[3], w["dW"], e["dW"])
    a.check_status()
    b.check_status()


@pytest.mark.parametrize("dtype", DTYPES)
def test_certain_tokens(dtype):
    # a vocabulary of one, and targets far above all others: losses of 0, not below
    for V, boost in ((1, 1.0), (200, 400.0)):
        x, W, target = make(150, 64, V, dtype, boost=0.0)
        x = (x.float() + boost * W[target].float()).to(dtype)
        loss, _, dx, dW = HeadLoss(150, W).cross_entropy(x, target)
        assert (loss >= 0).all() and float(loss.max()) <= 1e-5
        assert float(dx.float().abs().max()) <= 1e-5
        assert (HeadLoss(60, W, backward=False).score(x[:60], target[:60])[0] >= 0).all()


def test_weights_changed_in_place_take_effect():
    x, W, target = make(64, 64, 300, BF16)
    head = HeadLoss(64, W)
    check(head, x, target)
    W.mul_(-1.5)
    check(head, x, target)


def test_weights_given_other_memory_take_effect():
    x, W, target = make(64, 64, 300, BF16)
    head = HeadLoss(64, W)
    check(head, x, target)
    W.data = W.data * -1.5
    check(head, x, target)
    with pytest.raises(ops.MoEError, match="dtype"):
        W.data = W.data.float()
        head.score(x, target)


@pytest.mark.parametrize("T,d,V", [(129, 1536, 640), (300, 1544, 300), (257, 1600, 1000), (400, 2560, 129),
                                   (1000, 2568, 9000), (200, 4104, 20000)])
def test_long_rows(T, d, V):
    # around the lengths from which sums leave the tensor cores in chunks, of which the
    # last may be short; column tiles of which half the warps have none
    x, W, target = make(T, d, V, BF16, seed=d)
    target[::5] = -1
    check(HeadLoss(T, W), x, target, mean=True)
    want, bound = reference(x, W, target)
    head = HeadLoss(T, W, backward=False)
    loss, lse = head.score(x, target)
    near("loss", loss, want["loss"], bound["loss"])
    near("lse", lse, want["lse"], bound["lse"])
    head.check_status()
