"""The whole layer for a few tokens against the layer's formulas in 64 bits.

Tolerance, per element of y: y is rounded once to its type (2^-24 or 2^-8 of
it).  Before that, with A = sum_j w_j (|W2| |a| + |b2|) and B = sum_j w_j |W2|
(|W1| |x| + |b1|) (|GELU'| <= 1.13), a sum of n fp32 products is off by about
sqrt(n) 2^-24 of the sum of their magnitudes, here taken eight times over for
the largest of many elements; the gate weights' relative error is of the same
kind.  In bf16 the hidden activations are held in 16 bits (2^-16 of A) and GELU
is evaluated to 1.5e-7 of |h| (within 2^-16 of B).  Tokens whose k-th and
(k+1)-th logit are closer than their rounding are left out."""
import math
import os
import subprocess
import sys

import pytest
import torch

from mixture_experts_layer_11_gb300 import ops, synth
from mixture_experts_layer_11_gb300.decode import FewTokenPass
from mixture_experts_layer_11_gb300.layer import LayerPass
from parity_util import topk_margin

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = torch.float64


def make(T, d, f, E, k, dtype, bias=True, residual=True, beta=None, seed=0):
    cfg = synth.MoEConfig("few", T=T, d=d, f=f, E=E, k=k, renorm=1, dtype=dtype)
    p = synth.make_inputs(cfg, seed=seed, device=DEV, random_bias=True)
    p["residual"] = p.pop("dy")
    if not residual:
        p["residual"] = None
    if not bias:
        p["b1"] = p["b2"] = None
    p["beta"] = None if beta is None else beta.to(DEV)
    return p


def plain(p, k, renorm):
    """y, its tolerance and which tokens are decided, from the formulas."""
    x = p["x"].to(D)
    T, d = x.shape
    E, f, _ = p["W1"].shape
    L = x @ p["Wg"].to(D).T
    if p["beta"] is not None:
        L = L + p["beta"].to(D)
    prob = torch.softmax(L, 1)
    idx = torch.sort(L, dim=1, descending=True, stable=True)[1][:, :k]
    w = prob.gather(1, idx)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    y = torch.zeros(T, d, dtype=D, device=DEV)
    if p["residual"] is not None:
        y += p["residual"].to(D)
    A, B = y.abs(), torch.zeros_like(y)
    for e in idx.unique().tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        W1, W2 = p["W1"][e].to(D), p["W2"][e].to(D)
        b1 = p["b1"][e].to(D) if p["b1"] is not None else torch.zeros(f, dtype=D, device=DEV)
        b2 = p["b2"][e].to(D) if p["b2"] is not None else torch.zeros(d, dtype=D, device=DEV)
        h = x[t] @ W1.T + b1
        a = 0.5 * h * (1 + torch.erf(h / math.sqrt(2.0)))
        we = w[t, j][:, None]
        y[t] += we * (a @ W2.T + b2)
        A[t] += we * (a.abs() @ W2.abs().T + b2.abs())
        B[t] += we * ((x[t].abs() @ W1.abs().T + b1.abs()) @ W2.abs().T)
    bf16 = p["x"].dtype == torch.bfloat16
    fp32 = 8.0 * math.sqrt(max(d, f)) * 2.0 ** -24
    tol = (2.0 ** -8 if bf16 else 2.0 ** -24) * y.abs() + fp32 * (A + B)
    if bf16:
        tol += 2.0 ** -16 * (A + B)
    margin = torch.from_numpy(topk_margin(L.cpu().numpy(), k)) if k < E else torch.full((T,), math.inf)
    # two logits closer than this may change places (equal ones go by index on both sides)
    decided = (margin > 1e-5 * float(L.abs().max())) | (margin == 0)
    return y, tol, decided.to(DEV)


def layer(p, k, renorm, T=None):
    return FewTokenPass(T or p["x"].shape[0], p["Wg"], p["W1"], p["b1"], p["W2"], p["b2"], k, renorm,
                        beta=p["beta"])


def check(got, p, k, renorm):
    y, tol, decided = plain(p, k, renorm)
    assert decided.float().mean() > 0.8
    err = (got.to(D) - y).abs()
    bad = (err > tol) & decided[:, None]
    assert torch.isfinite(got).all()
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / tol)[decided].max()):.2f} of the tolerance")


SHAPES = [  # T, d, f, E, k
    (1, 8, 8, 1, 1), (1, 64, 128, 4, 1), (4, 64, 128, 4, 1), (2, 72, 200, 5, 2), (64, 8, 8, 256, 16),
    (63, 136, 120, 3, 3), (64, 128, 264, 2, 1), (33, 768, 264, 16, 2), (1, 1000, 2056, 7, 5),
    (16, 512, 1024, 8, 2), (17, 512, 1024, 64, 8), (64, 256, 640, 8, 8), (8, 2048, 128, 128, 8),
    (3, 128, 4096, 6, 1), (48, 4096, 64, 32, 16), (1, 4096, 1024, 128, 8), (64, 1024, 512, 128, 8),
    (5, 24, 1000, 1, 1), (9, 320, 320, 33, 4)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_layer(shape, dtype):
    T, d, f, E, k = shape
    p = make(T, d, f, E, k, dtype, seed=T + d)
    fp = layer(p, k, 1)
    check(fp.forward(p["x"], p["residual"]), p, k, 1)
    assert int(fp.status.item()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias,residual,renorm", [(False, False, 0), (True, False, 0), (False, True, 1)])
def test_options(dtype, bias, residual, renorm):
    p = make(13, 384, 512, 12, 3, dtype, bias, residual, synth.zipf_logit_bias(12, 1.2, 2.0))
    check(layer(p, 3, renorm).forward(p["x"], p["residual"]), p, 3, renorm)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 15, 16, 17, 31, 32, 33, 64])
def test_every_token_at_one_expert(dtype, T):
    # expert 5 of 8 takes all tokens, the others none; then a second one as well
    beta = torch.zeros(8)
    beta[5] = 1e4
    p = make(T, 256, 384, 8, 1, dtype, beta=beta, seed=T)
    check(layer(p, 1, 0).forward(p["x"], p["residual"]), p, 1, 0)
    beta[7] = 9e3
    p = make(T, 256, 384, 8, 2, dtype, beta=beta, seed=T)
    check(layer(p, 2, 0).forward(p["x"], p["residual"]), p, 2, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_logits_go_to_the_lower_expert(dtype):
    p = make(9, 128, 64, 40, 3, dtype)
    p["Wg"] = p["Wg"][:1].expand(40, -1).contiguous()   # all logits of a token are equal
    got = layer(p, 3, 1).forward(p["x"], p["residual"])
    y, tol, _ = plain(p, 3, 1)
    # experts 0, 1, 2 at weight 1/3 each
    q = dict(p, Wg=p["Wg"], beta=torch.tensor([0.0] * 3 + [-1e4] * 37, device=DEV))
    y, tol, _ = plain(q, 3, 1)
    assert ((got.to(D) - y).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_is_not_chosen_does_not_matter(dtype):
    # NaN and infinity in the weights of experts without tokens
    p = make(6, 136, 264, 16, 2, dtype)
    fp = layer(p, 2, 1)
    first = fp.forward(p["x"], p["residual"]).clone()
    idx = torch.sort(p["x"].double() @ p["Wg"].double().T, 1, descending=True)[1][:, :2]
    for e in range(16):
        if not (idx == e).any():
            p["W1"][e] = math.nan
            p["W2"][e] = math.inf
            p["b1"][e] = math.nan
            p["b2"][e] = -math.inf
    assert torch.equal(fp.forward(p["x"], p["residual"]), first)
    assert int(fp.status.item()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_non_finite_logits_are_reported_and_stay_with_their_token(dtype, bad):
    p = make(7, 64, 128, 4, 2, dtype)
    fp = layer(p, 2, 1)
    good = fp.forward(p["x"], p["residual"]).clone()
    p["x"][3, 5] = bad
    got = fp.forward(p["x"], p["residual"])
    torch.cuda.synchronize()
    assert int(fp.status.item()) == ops.MOE_ERR_NONFINITE
    keep = torch.arange(7, device=DEV) != 3
    # the other tokens' values do not change (their experts' rows do, so not their bits)
    _, tol, _ = plain(make(7, 64, 128, 4, 2, dtype), 2, 1)
    assert ((got.to(D) - good.to(D)).abs() <= 2 * tol)[keep].all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 768, 512, 8, 2), (37, 512, 768, 24, 4)])
def test_same_bits_every_time_whatever_the_workspace_holds(dtype, shape):
    T, d, f, E, k = shape
    p = make(T, d, f, E, k, dtype)
    fp = layer(p, k, 1)
    first = fp.forward(p["x"], p["residual"]).clone()
    for fill in (0xFF, 0x00, 0x7F):
        fp.ws.fill_(fill)
        for _ in range(3):
            assert torch.equal(fp.forward(p["x"], p["residual"]), first)
    assert int(fp.status.item()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_fewer_tokens_than_room_and_outputs_in_place(dtype):
    p = make(50, 264, 384, 16, 2, dtype)
    fp = layer(p, 2, 1)
    for t in (1, 2, 16, 49, 50):
        q = dict(p, x=p["x"][:t], residual=p["residual"][:t])
        check(fp.forward(q["x"], q["residual"]), q, 2, 1)
        out = q["residual"].clone()
        same = fp.forward(q["x"], q["residual"]).clone()
        fp.forward(q["x"], out, out=out)
        assert torch.equal(out, same)
    # nothing outside y is written
    guard = torch.full((60, 264), 7.0, dtype=p["x"].dtype, device=DEV)
    fp.forward(p["x"][:20], out=guard[20:40])
    assert (guard[:20] == 7).all() and (guard[40:] == 7).all() and not (guard[20:40] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_another_stream_and_a_graph(dtype):
    p = make(5, 256, 512, 8, 2, dtype)
    fp = layer(p, 2, 1)
    want = fp.forward(p["x"], p["residual"]).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp.y.zero_()
        fp.forward(p["x"], p["residual"])
    side.synchronize()
    assert torch.equal(fp.y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp.forward(p["x"], p["residual"])
    for seed in (3, 4):
        q = make(5, 256, 512, 8, 2, dtype, seed=seed)
        p["x"].copy_(q["x"])
        g.replay()
        check(fp.y, p, 2, 1)
    assert int(fp.status.item()) == 0


def test_two_layers_on_two_streams_at_once():
    p = [make(24, 512, 1024, 32, 4, "bf16", seed=s) for s in (1, 2)]
    fp = [layer(q, 4, 1) for q in p]
    want = [a.forward(q["x"], q["residual"]).clone() for a, q in zip(fp, p)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for a, q, s in zip(fp, p, streams):
            with torch.cuda.stream(s):
                a.forward(q["x"], q["residual"])
    torch.cuda.synchronize()
    for a, y in zip(fp, want):
        assert torch.equal(a.y, y) and int(a.status.item()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beside_kernels_that_hold_most_of_the_gpu(dtype):
    # its blocks come to run a few at a time, and take over the shares of those that do not
    p = make(40, 512, 1024, 32, 2, dtype)
    fp = layer(p, 2, 1)
    want = fp.forward(p["x"], p["residual"]).clone()
    big = torch.randn(8192, 8192, device=DEV, dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(3):
                torch.matmul(big, big)
        for _ in range(10):
            assert torch.equal(fp.forward(p["x"], p["residual"]), want)
        torch.cuda.synchronize()
    assert int(fp.status.item()) == 0


def test_right_behind_the_kernels_that_make_its_inputs():
    # the launches overlap the end of the kernel before them, not its results
    p = make(3, 256, 512, 8, 2, "bf16")
    fp = layer(p, 2, 1)
    xs = torch.randn(50, 3, 256, device=DEV).to(torch.bfloat16)
    want = [fp.forward(x, x).clone() for x in xs]
    out = torch.empty_like(xs)
    x = torch.empty_like(xs[0])
    for i in range(50):
        x.copy_(xs[i])
        out[i].copy_(fp.forward(x, x))
    assert torch.equal(out, torch.stack(want))


@pytest.mark.parametrize("name", ["tiny_f32", "moe_s_bf16"])
def test_agrees_with_the_layer_on_batches(name):
    cfg = synth.CONFIGS[name].scaled(T=64)
    p = synth.make_inputs(cfg, seed=5, device=DEV, random_bias=True)
    lp = LayerPass(64, cfg.d, cfg.f, cfg.E, cfg.k, cfg.torch_dtype, cfg.renorm)
    y = lp.forward(p["x"], p["Wg"], p["W1"], p["b1"], p["W2"], p["b2"])
    fp = FewTokenPass(64, p["Wg"], p["W1"], p["b1"], p["W2"], p["b2"], cfg.k, cfg.renorm)
    got = fp.forward(p["x"])
    scale = float(y.float().abs().max())
    assert float((got.float() - y.float()).abs().max()) <= (1e-5 if name == "tiny_f32" else 2e-2) * scale


def test_weights_beyond_32_bit_offsets():
    # 256 x 4096 x 4096 elements a matrix; the tokens go to the last two experts
    T, d, f, E = 3, 4096, 4096, 256
    W1 = torch.empty(E, f, d, dtype=torch.bfloat16, device=DEV)
    W2 = torch.empty(E, d, f, dtype=torch.bfloat16, device=DEV)
    beta = torch.full((E,), -1e4)
    beta[-2:] = 0
    small = make(T, d, f, 2, 2, "bf16")
    W1[-2:], W2[-2:] = small["W1"], small["W2"]
    Wg = torch.zeros(E, d, dtype=torch.bfloat16, device=DEV)
    Wg[-2:] = small["Wg"]
    fp = FewTokenPass(T, Wg, W1, None, W2, None, 2, 1, beta=beta.to(DEV))
    small["b1"] = small["b2"] = None
    check(fp.forward(small["x"], small["residual"]), small, 2, 1)


SHORT_WAIT = """
import torch
from mixture_experts_layer_11_gb300 import ops, synth
from mixture_experts_layer_11_gb300.decode import FewTokenPass
cfg = synth.MoEConfig("few", T=16, d=2048, f=4096, E=16, k=2, renorm=1, dtype={dtype!r})
p = synth.make_inputs(cfg, device="cuda")
fp = FewTokenPass(16, p["Wg"], p["W1"], p["b1"], p["W2"], p["b2"], 2, 1)
for _ in range(3):
    fp.status.zero_()
    fp.forward(p["x"])
    torch.cuda.synchronize()
    print(int(fp.status.item()))
assert int(torch.arange(10, device="cuda").sum()) == 45
"""


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_waits_that_run_out_are_reported(dtype):
    # 3 us: less than the second product waits for the first, so the call gives up,
    # says so, ends, and leaves the context usable
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SHORT_WAIT.format(dtype=dtype)], cwd=root, timeout=120,
                       env=dict(os.environ, MOE_WAIT_TIMEOUT_NS="3000"), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == [str(ops.MOE_ERR_TIMEOUT)] * 3


def test_refusals():
    p = make(4, 64, 128, 4, 2, "bf16")
    fp = layer(p, 2, 1)
    with pytest.raises(ValueError):
        fp.forward(torch.zeros(5, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        fp.forward(p["x"], p["residual"][:2])
    with pytest.raises(ops.MoEError):
        fp.forward(p["x"].float())
    with pytest.raises(ops.MoEError):
        fp.forward(p["x"].t().contiguous().t())
    with pytest.raises(ops.MoEError):
        fp.forward(p["x"].cpu())
    with pytest.raises(ops.MoEError):
        layer(dict(p, b1=p["b1"].float()), 2, 1)
