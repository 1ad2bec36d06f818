"""Cases, plain forms and 64-bit values of the operators between a model's last
hidden states and its training signal, over a vocabulary head W [V,d] whose
logits x W^T are never kept (``head.HeadLoss``):

``score``    log-probabilities of given tokens (as losses) and the log-sum-exp of
             each row: what scoring, evaluation and verification read;
``ce``       softmax cross entropy against target tokens, with the gradients of
             its mean with respect to the hidden states and the head;
``distill``  the divergence of the student's distribution from a teacher's top
             logits at a temperature, with the same gradients.

Widths are those of the workloads in ``synth.CONFIGS``; vocabularies, lists and
batches are general ones.
"""
import math
import random

import torch

own = False

# Widths (d) of the repository's workloads.
TINY, MOE_S, MOE_L, LONGCTX = 64, 768, 2048, 4096

SPAN = 512                            # tokens of a padded sequence
MOST = 4096 * 131072 * 4096           # T * V * d of the largest bf16 case
MOST_F32 = 1000 * 8009 * 768 * 4      # ... of the largest drawn in fp32
MOST_LOGITS = 4096 * 131072           # T * V of the largest case


def listed():
    return [
        # one new token's log-probability during decoding: latency, then the head's bytes
        dict(name="score_t1", op="score", T=1, d=MOE_S, V=50257, dtype="bf16", ignored=0.0),
        # a batch of an odd number of users, the widest head: the head's bytes
        dict(name="score_t13", op="score", T=13, d=LONGCTX, V=131072, dtype="bf16", ignored=0.0),
        # a small fp32 model's scores of a few sentences' tokens
        dict(name="score_f32_t33", op="score", T=33, d=MOE_S, V=32000, dtype="f32", ignored=0.0),
        # perplexity of a long text: products of long batches
        dict(name="score_t8191", op="score", T=8191, d=MOE_L, V=65536, dtype="bf16", ignored=0.0),
        # one training step's loss of the smallest fp32 model: all latency
        dict(name="ce_tiny_f32", op="ce", T=256, d=TINY, V=1000, dtype="f32", ignored=0.0, weighted=False),
        # the same of a middle-sized fp32 model, odd sizes
        dict(name="ce_f32", op="ce", T=1000, d=MOE_S, V=8009, dtype="f32", ignored=0.125, weighted=False),
        # fine-tuning on one short answer: the head's bytes, read and written
        dict(name="ce_t33", op="ce", T=33, d=MOE_L, V=32000, dtype="bf16", ignored=0.0, weighted=False),
        # a training step over padded sequences, odd vocabulary
        dict(name="ce_moe_s", op="ce", T=8192, d=MOE_S, V=50257, dtype="bf16", ignored=0.3, weighted=False),
        # the widest head: the largest products
        dict(name="ce_longctx", op="ce", T=4096, d=LONGCTX, V=131072, dtype="bf16", ignored=0.0, weighted=False),
        # a small fp32 student
        dict(name="distill_tiny_f32", op="distill", T=256, d=TINY, V=1000, dtype="f32", ignored=0.125, weighted=False,
             K=8, tau=1.0),
        # a student with a teacher's 64 best tokens, softened
        dict(name="distill_moe_s", op="distill", T=4096, d=MOE_S, V=50257, dtype="bf16", ignored=0.0, weighted=False,
             K=64, tau=2.0),
        # weighted tokens, padding, an odd batch and vocabulary
        dict(name="distill_moe_l", op="distill", T=5001, d=MOE_L, V=100003, dtype="bf16", ignored=0.1, weighted=True,
             K=32, tau=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = dict(op=rng.choice(["score", "ce", "ce", "distill", "distill"]), T=_log(rng, 1, 16384),
                 d=8 * _log(rng, 8, 512), V=_log(rng, 512, 131072), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]),
                 ignored=rng.choice([0.0, 0.0, rng.uniform(0.0, 0.6)]))
        if c["op"] != "score":
            c["weighted"] = rng.random() < 0.3
        if c["op"] == "distill":
            c.update(K=_log(rng, 1, 128), tau=rng.choice([1.0, 1.0, 2.0, rng.uniform(0.5, 4.0)]))
        cost = c["T"] * c["V"] * c["d"]
        if cost <= (MOST_F32 if c["dtype"] == "f32" else MOST) and c["T"] * c["V"] <= MOST_LOGITS:
            return c


# ---- inputs ------------------------------------------------------------------

def _kept(c):
    """Tokens of each span of SPAN that have a target; the rest is padding."""
    return SPAN - int(c["ignored"] * SPAN)


def _live(c):
    """Tokens with a target."""
    return c["T"] // SPAN * _kept(c) + min(c["T"] % SPAN, _kept(c))


def _inputs(c, seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    T, d, V = c["T"], c["d"], c["V"]

    # rows of the head have a norm of about 1, drawn a slice at a time
    W = torch.empty(V, d, dtype=dt, device=device)
    for part in W.split(8192):
        part.copy_(torch.randn(part.shape, generator=g, device=device) * d ** -0.5)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=device)

    # frequent tokens have small indices
    target = (V * uniform(T) ** 3).long().clamp_(max=V - 1)
    padding = torch.arange(T, device=device) % SPAN >= _kept(c)
    # hidden states with logits of standard deviation 2; the target's is raised by 0
    # (a token the model did not expect) to 14 (one it is sure of)
    x = 2.0 * torch.randn(T, d, generator=g, device=device)
    x += 14.0 * uniform(T, 1) * W[target].float()
    s = dict(c, W=W, x=x.to(dt), target=target.masked_fill(padding, -1))
    if c["op"] != "score":
        s["weight"] = 0.5 + uniform(T) if c["weighted"] else None
    if c["op"] == "distill":
        K = c["K"]
        # the teacher's K tokens: the target first, then others, none twice; logits
        # fall from 8; lists of some tokens are shorter
        gap = max(1, (V - 1) // K)
        steps = torch.randint(1, gap + 1, (T, K), generator=g, device=device)
        steps[:, 0] = 0
        idx = (target[:, None] + steps.cumsum(1)) % V
        logits = 8.0 - 10.0 * uniform(T, K).sort(1).values + 0.5 * torch.randn(T, K, generator=g, device=device)
        length = K - (uniform(T) ** 4 * K).long()
        absent = (torch.arange(K, device=device)[None] >= length[:, None]) | padding[:, None]
        s.update(idx=idx.masked_fill(absent, -1), logits=logits)
        del s["target"]
    return s


def prepare(c, seed):
    s = _inputs(c, seed)
    if own:
        from mixture_experts_layer_11_gb300.head import HeadLoss
        s["head"] = HeadLoss(c["T"], s["W"], entries=c.get("K", 1), backward=c["op"] != "score")
    return s


# ---- one pass ------------------------------------------------------------------

def _softmax_parts(x, W, live, tau):
    """Logits over the temperature in fp32 and their exponentials, sum and log-sum-exp."""
    x = torch.where(live[:, None], x.float(), 0.0)
    z = x @ W.float().T
    if tau != 1.0:
        z /= tau
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    return x, z, e, total, (top + torch.log(total))[:, 0]


def _gradients(s, x, G, live, factor):
    """dx and dW from the gradient of the logits up to a factor a row."""
    row = live * factor / live.sum().clamp(min=1)
    if s["weight"] is not None:
        row = row * s["weight"]
    G *= row[:, None]
    return (G @ s["W"].float()).to(s["x"].dtype), (G.T @ x).to(s["W"].dtype)


def _ce_plain(s):
    target = s["target"]
    live = target >= 0
    safe = target.clamp(min=0)
    x, z, e, total, lse = _softmax_parts(s["x"], s["W"], live, 1.0)
    rows = torch.arange(len(target), device=target.device)
    out = dict(loss=torch.where(live, lse - z[rows, safe], 0.0), lse=torch.where(live, lse, 0.0))
    if s["op"] == "ce":
        G = e.div_(total)
        G[rows, safe] -= 1.0
        out["dx"], out["dW"] = _gradients(s, x, G, live, 1.0)
    return out


def _distill_plain(s):
    idx, tau = s["idx"], s["tau"]
    present = idx >= 0
    live = present.any(1)
    safe = idx.clamp(min=0)
    t = torch.where(present, s["logits"] / tau, float("-inf"))
    top = torch.where(live, t.amax(1), 0.0)[:, None]
    q = torch.exp(t - top)
    mass = torch.where(live[:, None], q.sum(1, keepdim=True), 1.0)
    log_q = torch.where(present, t - top - torch.log(mass), 0.0)
    q = q / mass
    x, z, e, total, lse = _softmax_parts(s["x"], s["W"], live, tau)
    term = q * (log_q - z.gather(1, safe) + lse[:, None])
    out = dict(loss=tau * tau * torch.where(present, term, 0.0).sum(1), lse=torch.where(live, lse, 0.0))
    G = e.div_(total)
    G.scatter_add_(1, safe, -q)
    out["dx"], out["dW"] = _gradients(s, x, G, live, tau)
    return out


def run(s):
    if not own:
        return _distill_plain(s) if s["op"] == "distill" else _ce_plain(s)
    if s["op"] == "score":
        loss, lse = s["head"].score(s["x"], s["target"])
        return dict(loss=loss, lse=lse)
    if s["op"] == "ce":
        loss, lse, dx, dW = s["head"].cross_entropy(s["x"], s["target"], weight=s["weight"], mean=True)
    else:
        loss, lse, dx, dW = s["head"].distill(s["x"], s["idx"], s["logits"], temperature=s["tau"],
                                              weight=s["weight"], mean=True)
    return dict(loss=loss, lse=lse, dx=dx, dW=dW)


# ---- what a pass cannot do without ------------------------------------------------

def work(c):
    T, d, V, n = c["T"], c["d"], c["V"], _live(c)
    size = 4 if c["dtype"] == "f32" else 2
    entries = 12 * T * c["K"] if c["op"] == "distill" else 8 * T
    if c["op"] == "score":
        return {"bytes": size * d * (V + n) + entries + 8 * T, "flops": 2.0 * n * d * V}
    return {"bytes": size * d * (2 * V + n + T) + entries + (4 * T if c["weighted"] else 0) + 8 * T,
            "flops": 6.0 * n * d * V}


# ---- the definition in 64 bits -------------------------------------------------

def exact(c, seed):
    if 6.0 * c["T"] * c["d"] * c["V"] > 1.5e13:
        return None                       # over about 15 seconds
    s = _inputs(c, seed)
    D = torch.float64
    W, T = s["W"].to(D), c["T"]
    dev = W.device
    tau = c.get("tau", 1.0)
    loss, lse = torch.zeros(T, dtype=D, device=dev), torch.zeros(T, dtype=D, device=dev)
    backward = c["op"] != "score"
    if backward:
        dx, dW = torch.zeros(T, c["d"], dtype=D, device=dev), torch.zeros_like(W)
    count = max(1, _live(c))
    for a in range(0, T, 1024):
        rows = slice(a, min(T, a + 1024))
        if c["op"] == "distill":
            idx = s["idx"][rows]
            has = (idx >= 0).any(1)
        else:
            has = s["target"][rows] >= 0
        at = torch.nonzero(has)[:, 0]
        if at.numel() == 0:
            continue
        x = s["x"][rows][at].to(D)
        logp = torch.log_softmax(x @ W.T / tau, 1)
        n = torch.arange(len(at), device=dev)
        if c["op"] == "distill":
            idx = idx[at]
            logit = (s["logits"][rows][at].to(D) / tau).masked_fill(idx < 0, -math.inf)
            logq = torch.log_softmax(logit, 1)
            q = logq.exp()
            own_logp = logp[n[:, None], idx.clamp(min=0)]
            loss[a + at] = tau ** 2 * torch.where(q > 0, q * (logq - own_logp), 0.0).sum(1)
            first = s["idx"][rows][at][:, 0]
        else:
            first = s["target"][rows][at]
            loss[a + at] = -logp[n, first]
        # log-sum-exp from one logit and its log-probability
        lse[a + at] = (x * W[first]).sum(1) / tau - logp[n, first]
        if backward:
            G = logp.exp_()
            if c["op"] == "distill":
                G.scatter_add_(1, idx.clamp(min=0), -q)
            else:
                G[n, first] -= 1.0
            G *= tau / count
            if s["weight"] is not None:
                G *= s["weight"][rows][at].to(D)[:, None]
            dx[a + at] = G @ W
            dW += G.T @ x
    out = dict(loss=loss, lse=lse)
    if backward:
        out.update(dx=dx, dW=dW)
    return out
