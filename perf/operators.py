"""Cases, plain forms and 64-bit values of the operators for serving a trained
layer and for closing its training step:

``few``   one whole MoE layer for a few tokens (1 to 64): router, top-k gate,
          experts, combine and an optional residual, as a decode step calls it
          (``decode.FewTokenPass``);
``norm``  the global norm of a list of gradients (``grads.GradClip.norm``);
``clip``  that norm, and the gradients scaled so that it is at most a bound,
          written to a second list of buffers (``grads.GradClip.clip``).

Sizes are those of the workloads in ``synth.CONFIGS`` and general ones.
"""
import math
import random

import numpy as np
import torch

own = False

# The layers of the repository's workloads, as (d, f, E, k, renorm, zipf s).
TINY = dict(d=64, f=128, E=4, k=1, renorm=0, zipf=0.0)
MOE_S = dict(d=768, f=3072, E=8, k=2, renorm=1, zipf=0.0)
SKEWED = dict(d=768, f=3072, E=64, k=1, renorm=0, zipf=1.2)
MOE_L = dict(d=2048, f=8192, E=16, k=2, renorm=1, zipf=0.0)
LONGCTX = dict(d=4096, f=1024, E=128, k=8, renorm=1, zipf=1.1)

MOST_WEIGHTS = 128 * 4096 * 1024      # E * d * f of the largest case
MOST_SLOTS = 512 * 4096 * 1024        # T * k * d * f of the largest case
MOST_GRADS = 2 * 128 * 4096 * 1024    # gradient elements of the largest case


def listed():
    return [
        # four users' next tokens through the smallest fp32 layer: all latency
        dict(name="few_tiny_f32_t4", op="few", T=4, dtype="f32", bias=True, residual=False, **TINY),
        # one user's next token
        dict(name="few_moe_s_t1", op="few", T=1, dtype="bf16", bias=True, residual=True, **MOE_S),
        dict(name="few_longctx_t1", op="few", T=1, dtype="bf16", bias=False, residual=True, **LONGCTX),
        # a batch of an odd number of users, experts of very unequal load, fp32
        dict(name="few_skewed_f32_t33", op="few", T=33, dtype="f32", bias=True, residual=False, **SKEWED),
        # an odd batch over few wide experts: almost every expert is read
        dict(name="few_moe_l_t13", op="few", T=13, dtype="bf16", bias=True, residual=False, **MOE_L),
        # the largest batch over few experts (many tokens an expert) ...
        dict(name="few_moe_s_t64", op="few", T=64, dtype="bf16", bias=True, residual=True, **MOE_S),
        # ... and over many, evenly loaded (few tokens an expert, all weights read)
        dict(name="few_longctx_t64", op="few", T=64, dtype="bf16", bias=False, residual=True,
             **dict(LONGCTX, zipf=0.0)),
        # the five gradients of the smallest layer: all latency
        dict(name="clip_tiny", op="clip", layout="layer", over=True, **TINY),
        # the five gradients of one layer, somewhat above the L2's size
        dict(name="clip_moe_s", op="clip", layout="layer", over=True, **MOE_S),
        # a model's many parameters, fp32 and bf16, as views of two flat buffers
        # with odd sizes, so that most begin off a 16-byte boundary
        dict(name="clip_ragged", op="clip", layout="ragged", tensors=211, most=3000001, sizes=7, over=True),
        # the norm alone, for a training log or a skipped step
        dict(name="norm_moe_l", op="norm", layout="layer", over=True, **MOE_L),
        # the largest layer's gradients
        dict(name="clip_longctx", op="clip", layout="layer", over=True, **LONGCTX),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        while True:
            c = dict(op="few", T=_log(rng, 1, 64), dtype=dtype, bias=rng.random() < 0.5,
                     residual=rng.random() < 0.5, d=8 * _log(rng, 8, 512), f=8 * _log(rng, 16, 1024),
                     E=_log(rng, 1, 128))
            c.update(k=rng.randint(1, min(8, c["E"])), renorm=rng.randint(0, 1),
                     zipf=rng.choice([0.0, 0.0, 1.1, 1.2]))
            size = c["d"] * c["f"] * (2 if dtype == "f32" else 1)
            if c["E"] * size <= MOST_WEIGHTS and c["T"] * c["k"] * size <= MOST_SLOTS:
                return c
    op = rng.choice(["clip", "clip", "norm"])
    over = rng.random() < 0.75
    if rng.random() < 0.5:
        while True:
            c = dict(op=op, layout="layer", over=over, d=8 * _log(rng, 8, 512), f=8 * _log(rng, 16, 1024),
                     E=_log(rng, 1, 128), k=1, renorm=0, zipf=0.0)
            if 2 * c["E"] * c["d"] * c["f"] + c["E"] * (2 * c["d"] + c["f"]) <= MOST_GRADS:
                return c
    return dict(op=op, layout="ragged", tensors=_log(rng, 1, 1000), most=_log(rng, 64, 3000000),
                sizes=rng.randint(0, 1 << 30), over=over)


# ---- inputs ------------------------------------------------------------------

def _generator(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _shift(c):
    """The layer's fixed logit shift 2 ln((e + 1)^-s), or None."""
    if not c["zipf"]:
        return None
    return torch.tensor([-2.0 * c["zipf"] * math.log(e + 1.0) for e in range(c["E"])])


def _layer(c, seed, device="cuda"):
    g = _generator(seed, device)
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16

    def normal(std, *shape):
        # drawn a slice at a time in fp32: the largest weights need no fp32 copy of all of them
        out = torch.empty(shape, dtype=dt, device=device)
        for part in out.view(shape[0], -1).split(16):
            part.copy_(torch.randn(part.shape, generator=g, device=device) * std)
        return out

    T, d, f, E = c["T"], c["d"], c["f"], c["E"]
    p = dict(x=normal(1.0, T, d), Wg=normal(d ** -0.5, E, d), W1=normal(d ** -0.5, E, f, d),
             W2=normal(f ** -0.5, E, d, f))
    p["b1"] = normal(0.1, E, f) if c["bias"] else None
    p["b2"] = normal(0.1, E, d) if c["bias"] else None
    p["residual"] = normal(1.0, T, d) if c["residual"] else None
    beta = _shift(c)
    p["beta"] = None if beta is None else beta.to(device)
    return p


def _sizes(c):
    """[(elements, bf16 or not)] of the case's gradients, in order."""
    if c["layout"] == "layer":
        d, f, E = c["d"], c["f"], c["E"]
        return [(E * d, False), (E * f * d, False), (E * f, False), (E * d * f, False), (E * d, False)]
    rng = random.Random(c["sizes"])
    return [(_log(rng, 1, c["most"]), rng.random() < 0.4) for _ in range(c["tensors"])]


def _gradients(c, seed, device="cuda"):
    """Two flat buffers (fp32, bf16) and the gradients, which are views of them."""
    g = _generator(seed, device)
    sizes = _sizes(c)
    flat, views, at = [], [], [0, 0]
    for half, dt in ((False, torch.float32), (True, torch.bfloat16)):
        flat.append(torch.empty(sum(n for n, h in sizes if h == half), dtype=dt, device=device))
    for n, h in sizes:
        v = flat[h][at[h]:at[h] + n]
        at[h] += n
        views.append(v)
    for buf in flat:
        for part in buf.split(1 << 26):
            part.copy_(torch.randn(part.shape, generator=g, device=device))
    # gradients of different parameters have different scales
    scale = 10.0 ** (torch.rand(len(views), generator=_generator(seed + 1, "cpu")) * 3.0 - 4.0)
    for v, s in zip(views, scale.tolist()):
        v.mul_(s)
    return flat, views, scale.tolist()


def _bound(c, sizes, scale):
    """A clipping bound below (over) or above the norm that these scales lead to."""
    norm = math.sqrt(sum(n * s * s for (n, _), s in zip(sizes, scale)))
    return (0.3 if c["over"] else 3.0) * norm


def prepare(c, seed):
    if c["op"] == "few":
        s = dict(c, **_layer(c, seed))
        if own:
            from mixture_experts_layer_11_gb300.decode import FewTokenPass
            s["layer"] = FewTokenPass(c["T"], s["Wg"], s["W1"], s["b1"], s["W2"], s["b2"],
                                      c["k"], c["renorm"], beta=s["beta"])
        return s
    flat, views, scale = _gradients(c, seed)
    s = dict(c, flat=flat, grads=views, bound=_bound(c, _sizes(c), scale))
    if c["op"] == "clip":
        s["out"] = [torch.empty_like(b) for b in flat]
        at, outs = [0, 0], []
        for n, h in _sizes(c):
            outs.append(s["out"][h][at[h]:at[h] + n])
            at[h] += n
        s["outs"] = outs
    if own:
        from mixture_experts_layer_11_gb300.grads import GradClip
        s["handle"] = GradClip(s["grads"], s.get("outs"))
    return s


# ---- one pass ------------------------------------------------------------------

def _few_plain(s):
    x = s["x"].float()
    logits = x @ s["Wg"].float().T
    if s["beta"] is not None:
        logits = logits + s["beta"]
    # the k largest logits, equal ones by their index
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :s["k"]], idx[:, :s["k"]]
    w = torch.exp(logits - top[:, :1])
    w = torch.exp(top - top[:, :1]) / w.sum(1, keepdim=True)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    h = (s["W1"][idx].float() @ x[:, None, :, None])[..., 0]          # [T, k, f]
    if s["b1"] is not None:
        h = h + s["b1"][idx].float()
    a = 0.5 * h * (1.0 + torch.erf(h * math.sqrt(0.5)))
    y = (s["W2"][idx].float() @ a[..., None])[..., 0]                 # [T, k, d]
    if s["b2"] is not None:
        y = y + s["b2"][idx].float()
    y = (w[..., None] * y).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _norm_plain(s):
    return torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()


def run(s):
    if s["op"] == "few":
        if own:
            return s["layer"].forward(s["x"], residual=s["residual"])
        return _few_plain(s)
    if s["op"] == "norm":
        return s["handle"].norm() if own else _norm_plain(s)
    if own:
        return [s["handle"].clip(s["bound"])] + s["out"]
    norm = _norm_plain(s)
    factor = torch.clamp(s["bound"] / norm, max=1.0)
    [o.copy_(g.float() * factor) for g, o in zip(s["grads"], s["outs"])]
    return [norm] + s["out"]


# ---- what a pass cannot do without ------------------------------------------------

def _touched(c):
    """Distinct experts that T tokens choose: counted on one draw of N(0,1) logits."""
    r = np.random.default_rng(1)
    logits = r.standard_normal((c["T"], c["E"]))
    shift = _shift(c)
    if shift is not None:
        logits = logits + shift.numpy()
    return len(np.unique(np.argsort(-logits, axis=1)[:, :c["k"]]))


def work(c):
    if c["op"] == "few":
        T, d, f, E, k = (c[n] for n in ("T", "d", "f", "E", "k"))
        size = 4 if c["dtype"] == "f32" else 2
        n = _touched(c)
        weights = n * 2 * d * f + (n * (d + f) if c["bias"] else 0) + E * d
        rows = T * d * (3 if c["residual"] else 2)
        return {"bytes": size * (weights + rows) + (4 * E if c["zipf"] else 0),
                "flops": 2.0 * T * E * d + 4.0 * T * k * d * f}
    sizes = _sizes(c)
    count = sum(n for n, _ in sizes)
    read = sum(n * (2 if h else 4) for n, h in sizes)
    if c["op"] == "norm":
        return {"bytes": read, "flops": 2.0 * count}
    return {"bytes": 2 * read, "flops": 3.0 * count}


# ---- the definition in 64 bits -------------------------------------------------

def exact(c, seed):
    if c["op"] == "few":
        p = _layer(c, seed)
        D = torch.float64
        x = p["x"].to(D)
        logits = torch.einsum("td,ed->te", x, p["Wg"].to(D))
        if p["beta"] is not None:
            logits = logits + p["beta"].to(D)
        prob = torch.softmax(logits, 1)
        y = torch.zeros_like(x) if p["residual"] is None else p["residual"].to(D)
        chosen = torch.zeros_like(prob)
        for t, row in enumerate(logits.cpu().numpy()):
            for e in np.lexsort((np.arange(c["E"]), -row))[:c["k"]]:
                chosen[t, int(e)] = prob[t, int(e)]
        if c["renorm"]:
            chosen = chosen / chosen.sum(1, keepdim=True)
        for e in range(c["E"]):
            rows = torch.nonzero(chosen[:, e])[:, 0]
            if rows.numel() == 0:
                continue
            h = x[rows] @ p["W1"][e].to(D).T
            if p["b1"] is not None:
                h = h + p["b1"][e].to(D)
            a = h * torch.special.ndtr(h)
            out = a @ p["W2"][e].to(D).T
            if p["b2"] is not None:
                out = out + p["b2"][e].to(D)
            y[rows] += chosen[rows, e][:, None] * out
        return y
    flat, views, scale = _gradients(c, seed)
    total = 0.0
    for v in views:
        for part in v.split(1 << 26):
            total += float((part.double() ** 2).sum())
    norm = math.sqrt(total)
    if c["op"] == "norm":
        return torch.tensor(norm, dtype=torch.float64)
    bound = _bound(c, _sizes(c), scale)
    factor = bound / norm if norm > bound else 1.0
    return [torch.tensor(norm, dtype=torch.float64)] + [b.double() * factor for b in flat]
