"""Losses over a vocabulary head where the logits over the temperature are large: up
to 2^113, of which fp32 holds 24 bits.  The logits are exact here (one nonzero column:
a power of two times at most 8 bits), so that the bounds are those of the softmax alone,
with u = 2^-24 and h = 2^-8 (bf16: half a step; fp32: 0):
 differences to the largest logit  exact, times log2(e) / temperature: 2 u of them
 lse        4 u of its size, and 2^-19 (sums, logarithm)
 loss       temperature^2 times: each term by 2^-20 and its q's share, 8 u |log q| (the
            exponent's rounding) and 2^-149 (fp32's last number); and 2^-18, as lse
 G          p by 2^-11 (exponentials as fp16) and 2^-16 (2 u of a difference of up to 64 bits,
            exponentials, sums) of it, 2^-40 of the block's largest, the teacher's by 2^-18; h
 dx, dW     as in head_util
"""
import pytest
import torch

from head_util import D, U, near
from mixture_experts_layer_11_gb300.head import HeadLoss

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def inputs(T, d, V, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.zeros(T, d, device="cuda")
    x[:, 0] = 2.0 ** (torch.arange(T, device="cuda") % 101).float()
    W = torch.zeros(V, d, device="cuda")
    W[:, 0] = torch.randint(-127, 128, (V,), generator=g, device="cuda") / 128
    # targets: the largest logit, the smallest, any
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[::3] = W[:, 0].argmax()
    target[1::7] = W[:, 0].argmin()
    idx = torch.randint(0, V, (T, 3), generator=g, device="cuda")
    idx[:, 0] = target
    return x.to(dtype), W.to(dtype), target, idx, torch.randn(T, 3, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,d,V", [(7, 8, 300), (120, 8, 300), (210, 8, 515), (210, 1600, 300), (202, 8, 10007)])
@pytest.mark.parametrize("tau", [None, 1e-4, 0.01])
def test_large_logits(T, d, V, tau, dtype):
    x, W, target, idx, logits = inputs(T, d, V, dtype, T + V)
    h = 2.0 ** -8 if dtype == BF16 else 0.0
    t = 1.0 if tau is None else tau
    x64, W64 = x.to(D), W.to(D)
    tf = float(torch.tensor(t, dtype=F32))              # what the call takes
    z = x64 @ W64.T / tf
    lse = torch.logsumexp(z, 1)
    if tau is None:
        at, logq = target[:, None], torch.zeros(T, 1, dtype=D, device="cuda")
    else:
        at, logq = idx, torch.log_softmax(logits.to(D) / tf, 1)
    q = logq.exp()
    Q = torch.zeros_like(z).scatter_add_(1, at, q)
    # (from the differences to the largest logit: the logits have no bits left below 1)
    top = z.amax(1, keepdim=True)
    gap = (top - z).gather(1, at)
    log_sum = torch.log(torch.exp(z - top).sum(1))
    logq = torch.where(q > 0, logq, 0.0)
    loss = tf * tf * ((q * (logq + gap)).sum(1) + log_sum)
    e_loss = q * (2.0 ** -20 + 8 * U * logq.abs()) * (gap + logq.abs()) + 2.0 ** -149 * gap
    e_loss = tf * tf * (e_loss.sum(1) + 2.0 ** -18)
    e_lse = 4 * U * lse.abs() + 2.0 ** -19
    p = torch.exp(z - top - log_sum[:, None])
    G = p - Q
    eG = p * (2.0 ** -11 + 2.0 ** -16) + 2.0 ** -40 + Q * 2.0 ** -18 + (Q > 0) * 2.0 ** -18
    eG = eG * (1 + h) + G.abs() * (h + 2 * U)
    dx, dW, aG = tf * (G @ W64), tf * (G.T @ x64), G.abs() + eG
    e_dx = tf * (eG @ W64.abs() + (V + 4) * 2 * U * (aG @ W64.abs())) * (1 + h) + dx.abs() * (h + 4 * U)
    e_dW = tf * (eG.T @ x64.abs() + (T + 4) * 2 * U * (aG.T @ x64.abs())) * (1 + h) + dW.abs() * (h + 4 * U)
    head, scores = HeadLoss(T, W, entries=3), HeadLoss(T, W, entries=3, backward=False)
    for o in (scores, head):
        if tau is None:
            got = o.score(x, target) if o is scores else o.cross_entropy(x, target)
        else:
            got = o.distill(x, idx, logits, temperature=t)
        near("loss", got[0], loss, e_loss)
        near("lse", got[1], lse, e_lse)
        o.check_status()
    near("dx", got[2], dx, e_dx)
    near("dW", got[3], dW, e_dW)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [5, 200])
def test_certain_tokens_of_large_logits(T, dtype):
    # the largest logit alone: a loss of 0 and gradients of 0, whatever its size
    x, W, _, _, _ = inputs(T, 8, 300, dtype, 1)
    W[:, 0] = -W[:, 0].abs()
    W[17, 0] = 1.0
    x[:, 0] = torch.maximum(x[:, 0], torch.tensor(2.0 ** 8, dtype=dtype, device="cuda"))
    target = torch.full((T,), 17, device="cuda")
    head = HeadLoss(T, W)
    loss, _, dx, dW = head.cross_entropy(x, target)
    assert not loss.any() and not dx.float().any() and not dW.float().any()
    assert not head.score(x, target)[0].any()
    head.check_status()
