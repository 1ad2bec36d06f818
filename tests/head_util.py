"""Losses over a vocabulary head in 64 bits, with bounds of what the kernels may be
off by, element by element.

Bounds, with u = 2^-24 (half a step of fp32) and h = 2^-8 (of bf16, 0 in fp32):
 logits     a sum of d products in fp32, rounded or cut off after each: at most
            2 d u sum_i |x_i W_vi| (a product of bf16 numbers is exact; one of fp32
            numbers is rounded within the fused operation), over the temperature;
            converting to bits and exponent another 4 u of the logit's size
 lse        no more than the largest of its logits' errors, and the sum's: 2^-19 of
            the sum (exponentials to 2^-21, sums of a block, of blocks), and rounding
 p          2 errors of logits as a factor, exp() to 2^-20
 E          bf16 calls hold the exponentials as fp16: 2^-11 of each and 2^-40 of
            their block's largest
 G          weight (p - q): the errors above, q to 2^-20, and h of the result
 dx, dW     sums of n products in fp32: (n + 4) 2 u sum |G W|, G's errors through the
            product, and h of the result
"""
import torch

U = 2.0 ** -24
D = torch.float64


def reference(x, W, target=None, idx=None, logits=None, temperature=1.0, weight=None, scale=1.0,
              mean=False):
    """dict of values and dict of bounds (loss, lse, dx, dW), 64 bits, CPU or GPU."""
    bf16 = x.dtype == torch.bfloat16
    h = 2.0 ** -8 if bf16 else 0.0
    T, d = x.shape
    V = W.shape[0]
    x64, W64 = x.to(D), W.to(D)
    Q = torch.zeros(T, V, dtype=D, device=x.device)       # the target distribution
    entropy = torch.zeros(T, dtype=D, device=x.device)    # sum q log q
    if target is not None:
        live = (target >= 0) & (target < V)
        Q[live, target[live]] = 1.0
        entries_err = torch.zeros(T, dtype=D, device=x.device)
    else:
        present = (idx >= 0) & (idx < V) & (logits != float("-inf"))
        live = present.any(1)
        t = (logits.to(D) / temperature).masked_fill(~present, float("-inf"))
        t[~live] = 0.0
        logq = torch.log_softmax(t, 1)
        q = torch.where(present, logq.exp(), 0.0)
        Q.scatter_add_(1, torch.where(present, idx, 0), q)
        entropy = torch.where(q > 0, q * logq, 0.0).sum(1)
        # the softmax of the entries, in fp32: their arguments, their sum
        size = torch.where(present & (q > 0), logq.abs(), 0.0)
        entries_err = (q * (2.0 ** -20 + 8 * U * size)).sum(1)
    x64 = torch.where(live[:, None], x64, 0.0)
    z = x64 @ W64.T / temperature
    lse = torch.logsumexp(z, 1)
    logp = z - lse[:, None]
    p = logp.exp()
    zero = torch.zeros_like(lse)
    loss = temperature ** 2 * (entropy - torch.where(Q > 0, Q * logp, 0.0).sum(1))
    ez = 2 * d * U * (x64.abs() @ W64.abs().T) / temperature + 4 * U * z.abs()
    e_lse = ez.amax(1) + 2.0 ** -19 + 8 * U * lse.abs()
    e_logp = ez + e_lse[:, None]
    e_loss = temperature ** 2 * ((Q * e_logp).sum(1) + entries_err
                                 + 8 * U * (Q * (logp.abs() + lse.abs()[:, None])).sum(1)
                                 + 136 * U * (entropy.abs() + (Q * logp.abs()).sum(1)))
    w = torch.ones_like(lse) if weight is None else weight.to(D)
    count = max(1, int(live.sum())) if mean else 1
    G = torch.where(live[:, None], w[:, None] * (p - Q), 0.0)
    blocks = torch.nn.functional.pad(p, (0, -V % 128)).view(T, -(-V // 128), 128).amax(2)
    largest = blocks.repeat_interleave(128, 1)[:, :V]
    eG = p * (torch.expm1(2 * e_logp) + 2.0 ** -19) + Q * 2.0 ** -19
    eG = eG + torch.where(Q > 0, entries_err[:, None] + 2.0 ** -22, 0.0)
    if bf16:
        eG = eG + p * 2.0 ** -11 + largest * 2.0 ** -40
    eG = torch.where(live[:, None], w.abs()[:, None] * eG, 0.0)
    eG = eG + G.abs() * (h + 2 * U) + eG * h
    f = scale * temperature / count
    # (padded rows of a last K block are exact zeros)
    dx, dW = f * (G @ W64), f * (G.T @ x64)
    aG = G.abs() + eG
    e_dx = abs(f) * (eG @ W64.abs() + (V + 4) * 2 * U * (aG @ W64.abs()))
    e_dW = abs(f) * (eG.T @ x64.abs() + (T + 4) * 2 * U * (aG.T @ x64.abs()))
    e_dx = e_dx * (1 + h) + dx.abs() * (h + 4 * U)
    e_dW32 = e_dW + dW.abs() * 4 * U
    e_dW = e_dW * (1 + h) + dW.abs() * (h + 4 * U)
    values = dict(loss=torch.where(live, loss, zero), lse=torch.where(live, lse, zero), dx=dx, dW=dW)
    bounds = dict(loss=torch.where(live, e_loss, zero), lse=torch.where(live, e_lse, zero), dx=e_dx,
                  dW=e_dW, dW32=e_dW32)
    return values, bounds


def near(name, got, want, bound):
    """Every element within its bound (and exact where that is 0)."""
    assert got.shape == want.shape, name
    off = (got.to(D) - want).abs()
    bad = ~(off <= bound + 1e-44)
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} elements, first {i}: "
                             f"{float(got[i])} for {float(want[i])} +- {float(bound[i])}")


def make(T, d, V, dtype, seed=0, device="cuda", spread=2.0, boost=8.0):
    """Hidden states, a head with rows of norm 1, and targets whose logits are raised."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    W = (torch.randn(V, d, generator=g, device=device) * d ** -0.5).to(dtype)
    target = torch.randint(0, V, (T,), generator=g, device=device)
    x = spread * torch.randn(T, d, generator=g, device=device)
    x += boost * torch.rand(T, 1, generator=g, device=device) * W[target].float()
    return x.to(dtype), W, target


def make_entries(T, K, V, target, seed=0, device="cuda", distinct=True):
    g = torch.Generator(device=device)
    g.manual_seed(seed + 77)
    idx = torch.randint(0, V, (T, K), generator=g, device=device)
    if distinct and V >= K:
        idx = torch.rand(T, V, generator=g, device=device).argsort(1)[:, :K].contiguous()
    idx[:, 0] = target
    logits = 3.0 * torch.randn(T, K, generator=g, device=device)
    return idx, logits
