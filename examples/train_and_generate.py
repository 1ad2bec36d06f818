"""Train one MoE layer on synthetic data, then serve it a few tokens at a time.

Training: ``LayerPass`` forward and backward on batches of tokens, the norm of
all five gradients clipped with ``GradClip``, a plain SGD step on fp32 master
weights.  Serving: ``FewTokenPass`` on the trained bf16 weights, its decode step
captured once in a CUDA graph and replayed for every new token.

    python examples/train_and_generate.py [--steps 60] [--tokens 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_layer_11_gb300.decode import FewTokenPass  # noqa: E402
from mixture_experts_layer_11_gb300.grads import GradClip  # noqa: E402
from mixture_experts_layer_11_gb300.layer import LayerPass  # noqa: E402

T, D, F, E, K = 4096, 256, 512, 8, 2     # tokens a batch, widths, experts, experts a token
BF16 = torch.bfloat16


def weights(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda std, *shape: torch.randn(shape, generator=g, device="cuda") * std  # noqa: E731
    zeros = lambda *shape: torch.zeros(shape, device="cuda")  # noqa: E731
    return [normal(D ** -0.5, E, D), normal(D ** -0.5, E, F, D), zeros(E, F),
            normal(F ** -0.5, E, D, F), zeros(E, D)]


def train(steps, max_norm=1.0, rate=0.5):
    """The trained (Wg, W1, b1, W2, b2) in bf16; prints the loss and the norm."""
    teacher = [w.to(BF16) for w in weights(1)]
    master = weights(2)
    params = [w.to(BF16) for w in master]
    layer = LayerPass(T, D, F, E, K, BF16, renorm=1)
    target = LayerPass(T, D, F, E, K, BF16, renorm=1)
    grads = [layer.dWg, layer.dW1, layer.db1, layer.dW2, layer.db2]
    clip = GradClip(grads)
    losses = []
    for step in range(steps):
        x = torch.randn(T, D, device="cuda").to(BF16)
        want = target.forward(x, *teacher)
        y = layer.forward(x, *params)
        diff = y.float() - want.float()
        losses.append(diff.square().mean())
        layer.backward((diff * (2.0 / T)).to(BF16), x, params[0], params[1], params[3])
        norm = clip.clip(max_norm)
        for m, p, g in zip(master, params, grads):
            m.sub_(g, alpha=rate)
            p.copy_(m)
        if step % 10 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {losses[-1].item():.4f}  gradient norm {norm.item():.3f}")
    layer.check_status()
    clip.check_status()
    return params, [float(v) for v in losses]


def generate(params, sequences, tokens):
    """`tokens` steps of x -> normalised (x + layer(x)) for some sequences at once;
    returns all states [tokens + 1, sequences, D]."""
    Wg, W1, b1, W2, b2 = params
    layer = FewTokenPass(sequences, Wg, W1, b1, W2, b2, K, renorm=1)
    x = torch.randn(sequences, D, device="cuda").to(BF16)

    def step():
        y = layer.forward(x, residual=x).float()
        x.copy_(y / y.square().mean(1, keepdim=True).sqrt())

    states = [x.clone()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()                                  # warm up, then start over
        x.copy_(states[0])
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(tokens):
        graph.replay()
        states.append(x.clone())
    layer.check_status()
    return torch.stack(states)


def check(params, states):
    """The largest difference, relative to the largest value, between the decode
    step and the batch layer on the same states."""
    x = states.reshape(-1, D).contiguous()
    batch = LayerPass(x.shape[0], D, F, E, K, BF16, renorm=1)
    want = batch.forward(x, *params).float()
    few = FewTokenPass(states.shape[1], *params, K, renorm=1)
    got = torch.cat([few.forward(s).clone() for s in states]).float()
    return float((got - want).abs().max() / want.abs().max())


def main(argv=None):
    a = argparse.ArgumentParser()
    a.add_argument("--steps", type=int, default=60)
    a.add_argument("--tokens", type=int, default=16)
    a.add_argument("--sequences", type=int, default=5)
    a = a.parse_args(argv)
    torch.manual_seed(0)
    params, losses = train(a.steps)
    states = generate(params, a.sequences, a.tokens)
    off = check(params, states)
    print(f"{a.tokens} tokens for {a.sequences} sequences; decode and batch differ by {off:.1e} of the largest value")
    return losses, states, off


if __name__ == "__main__":
    main()
