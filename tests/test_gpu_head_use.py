"""Losses over a vocabulary head as they are used: behind the layer and in front of
its backward pass, with clipping, beside other streams, over many tokens, and when a
wait inside a kernel runs out."""
import os
import sys
import time

import pytest
import torch

from head_util import make, make_entries, near, reference
from mixture_experts_layer_11_gb300 import ops, synth
from mixture_experts_layer_11_gb300.decode import FewTokenPass
from mixture_experts_layer_11_gb300.grads import GradClip
from mixture_experts_layer_11_gb300.head import HeadLoss
from mixture_experts_layer_11_gb300.layer import LayerPass

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = [F32, BF16]


def layer_inputs(dtype, T=300, d=128, f=192, E=4, k=2):
    cfg = synth.MoEConfig("t", T=T, d=d, f=f, E=E, k=k, renorm=1, dtype="f32" if dtype == F32 else "bf16")
    inp = {n: (v.cuda() if v is not None else None) for n, v in synth.make_inputs(cfg, seed=5, random_bias=True).items()}
    return cfg, inp


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_training_step(dtype):
    """layer -> loss -> layer's backward -> clipping, and the same step from a graph."""
    cfg, p = layer_inputs(dtype)
    V = 777
    _, W, target = make(cfg.T, cfg.d, V, dtype)
    target[::6] = -1
    lp = LayerPass(cfg.T, cfg.d, cfg.f, cfg.E, cfg.k, dtype, cfg.renorm)
    head = HeadLoss(cfg.T, W, dW=torch.empty(V, cfg.d, device="cuda"))
    grads = [lp.dWg, lp.dW1, lp.db1, lp.dW2, lp.db2, head.dW]
    clip = GradClip(grads)

    def step():
        y = lp.forward(p["x"], p["Wg"], p["W1"], p["b1"], p["W2"], p["b2"])
        loss, _, dy, _ = head.cross_entropy(y, target, mean=True)
        lp.backward(dy, p["x"], p["Wg"], p["W1"], p["W2"])
        return y, loss, dy, clip.clip(1e-3)

    y, loss, dy, norm = step()
    want, bound = reference(y, W, target, mean=True)
    near("loss", loss, want["loss"], bound["loss"])
    near("dy", dy, want["dx"], bound["dx"])
    # the gradients were scaled in place to a norm of 1e-3 (or were below it)
    total = torch.sqrt(sum((v.double() ** 2).sum() for v in grads))
    assert float(total) <= 1e-3 * (1 + 1e-5)
    scale = min(1.0, 1e-3 / float(norm))
    near("dW", head.dW, want["dW"] * scale, (bound["dW32"] + 1e-5 * want["dW"].abs()) * scale)
    eager = [v.clone() for v in (loss, dy, norm, *grads)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for g in grads:
        g.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, (loss, dy, norm, *grads)))
    for part in (lp, head, clip):
        part.check_status()


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_of_decoded_tokens(dtype):
    cfg, p = layer_inputs(dtype)
    _, W, target = make(40, cfg.d, 501, dtype)
    few = FewTokenPass(40, p["Wg"], p["W1"], p["b1"], p["W2"], p["b2"], cfg.k, cfg.renorm)
    y = few.forward(p["x"][:40], residual=p["x"][:40])
    scores = HeadLoss(40, W, backward=False)
    for t in (1, 7, 40):
        loss, lse = scores.score(y[:t], target[:t])
        want, bound = reference(y[:t], W, target[:t])
        near("loss", loss, want["loss"], bound["loss"])
        near("lse", lse, want["lse"], bound["lse"])
    few.check_status()
    scores.check_status()


def test_the_examples_steps():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_and_generate as example
    torch.manual_seed(0)
    losses, (y, W, idx, logits), (dx, dW) = example.train_tokens(3, 701)
    assert len(losses) == 3
    some = torch.arange(0, example.T, 16, device="cuda")
    want, bound = reference(y[some], W, idx=idx[some], logits=logits[some], temperature=2.0,
                            scale=1.0 / example.T)
    near("dx", dx[some], want["dx"], bound["dx"])
    want, bound = reference(y, W, idx=idx, logits=logits, temperature=2.0, mean=True)
    near("dW", dW, want["dW"], bound["dW32"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,V", [(16384, 16, 70), (16385, 16, 70), (20001, 24, 131), (70001, 8, 40)])
def test_many_tokens(T, d, V, dtype):
    # counted once (above 16384 tokens), in more than one round (above 65536 live ones)
    x, W, target = make(T, d, V, dtype, seed=T)
    target[::7] = -1
    target[T // 2:T // 2 + 1000] = -1
    head = HeadLoss(T, W, entries=3)
    loss, lse, dx, dW = head.cross_entropy(x, target, mean=True)
    want, bound = reference(x, W, target, mean=True)
    for k, v in (("loss", loss), ("lse", lse), ("dx", dx), ("dW", dW)):
        near(k, v, want[k], bound["dW32" if k == "dW" and dtype == F32 else k])
    scores = HeadLoss(T, W, backward=False)
    loss, lse = scores.score(x, target)
    near("loss", loss, want["loss"], bound["loss"])
    near("lse", lse, want["lse"], bound["lse"])
    idx, logits = make_entries(T, 3, V, target.clamp(min=0))
    idx[target < 0] = -1
    loss, _, dx, dW = head.distill(x, idx, logits)
    want, bound = reference(x, W, idx=idx, logits=logits)
    near("loss", loss, want["loss"], bound["loss"])
    near("dx", dx, want["dx"], bound["dx"])
    near("dW", dW, want["dW"], bound["dW32" if dtype == F32 else "dW"])
    head.check_status()


@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_beyond_32_bits(dtype):
    # 17000 rows of 131072 probabilities: 2.2e9 of them; the last rows against the formulas
    T, d, V = 17000, 8, 131072
    x, W, target = make(T, d, V, dtype)
    head = HeadLoss(T, W, piece=T)
    loss, lse, dx, _ = head.cross_entropy(x, target)
    want, bound = reference(x[-200:], W, target[-200:])
    for k, v in (("loss", loss), ("lse", lse), ("dx", dx)):
        near(k, v[-200:], want[k], bound[k])
    head.check_status()


def test_two_objects_on_two_streams():
    jobs = []
    for i, dtype in enumerate((BF16, F32, BF16)):
        x, W, target = make(400 + 64 * i, 128, 900 + i, dtype, seed=i)
        want = [v.clone() for v in HeadLoss(x.shape[0], W).cross_entropy(x, target)]
        jobs.append((HeadLoss(x.shape[0], W), x, target, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for head, x, target, _, stream in jobs:
            with torch.cuda.stream(stream):
                head.cross_entropy(x, target)
    torch.cuda.synchronize()
    for head, _, _, want, _ in jobs:
        got = (head.loss, head.lse, head.dx, head.dW)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        head.check_status()


def test_tensors_the_library_cannot_check_are_refused():
    x, W, target = make(32, 64, 100, BF16)
    idx, logits = make_entries(32, 4, 100, target)
    head = HeadLoss(32, W, entries=4)
    with pytest.raises(ops.MoEError):
        HeadLoss(32, W.t().contiguous().t())
    for call in (lambda: head.cross_entropy(x.float(), target), lambda: head.cross_entropy(x, target.int()),
                 lambda: head.cross_entropy(x, target, weight=torch.ones(32, device="cuda", dtype=BF16)),
                 lambda: head.cross_entropy(x.t().contiguous().t(), target),
                 lambda: head.cross_entropy(x, target.repeat_interleave(2)[::2]),
                 lambda: head.distill(x, idx, logits.double()), lambda: head.distill(x, idx.int(), logits),
                 lambda: head.distill(x, idx[:, ::2], logits[:, ::2]),
                 lambda: head.distill(x, idx, logits, temperature=0.0)):
        with pytest.raises(ops.MoEError):
            call()
    head.check_status()


@pytest.mark.parametrize("T,d,hook", [(T, 192, hook) for T in (100, 600) for hook in ("0:0:1", "0:1:0", "2:0:1", "2:1:0")]
                         + [(300, 2048, "0:0:20"), (300, 2048, "0:1:3")])
def test_waits_that_run_out(T, d, hook, monkeypatch):
    """With MOE_DEBUG_HEAD_WITHHOLD the producer of one unit issues nothing from a K
    block on (no copy is left in flight for it): the waits on that stage run out after
    1 s, the CTA waits for its copies, frees tensor memory and reports.  Afterwards the
    same call gives the same bits as before."""
    x, W, target = make(T, d, 1500, BF16)
    head = HeadLoss(T, W)
    good = [v.clone() for v in head.cross_entropy(x, target)]
    head.check_status()
    monkeypatch.setenv("MOE_DEBUG_HEAD_WITHHOLD", hook)
    began = time.time()
    head.cross_entropy(x, target)
    torch.cuda.synchronize()
    took = time.time() - began
    with pytest.raises(ops.MoEError) as e:
        head.check_status()
    assert e.value.code == ops.MOE_ERR_TIMEOUT and 0.9 < took < 20.0
    monkeypatch.delenv("MOE_DEBUG_HEAD_WITHHOLD")
    again = head.cross_entropy(x, target)
    assert all(torch.equal(a, b) for a, b in zip(good, again))
    head.check_status()
