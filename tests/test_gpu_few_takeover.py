"""Shares of few_experts_kernel whose own block cannot run are taken over.

The kernel has a block for every SM, and a block needs all of an SM's shared
memory.  Here other kernels, of one thread each, hold some SMs from before the
call until after it: as many blocks cannot run before others have ended, and
none ends before all shares are done.  So a call that is complete while they
still run has taken shares over; its result must have the same bits."""
import pytest
import torch

from mixture_experts_layer_11_gb300 import synth
from mixture_experts_layer_11_gb300.decode import FewTokenPass

pytestmark = pytest.mark.gpu
DEV = "cuda"
CYCLES, AHEAD = 60_000_000, 6_000_000   # some 30 ms, and 3 ms


def event():
    return torch.cuda.Event(enable_timing=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("held", [1, 6, 120])
def test_shares_of_blocks_that_cannot_run(dtype, held):
    # 120: fewer blocks run than there are tokens, so that their gate is not shared out either
    T, d, f, E, k = 40, 512, 1024, 32, 2
    cfg = synth.MoEConfig("few", T=T, d=d, f=f, E=E, k=k, renorm=1, dtype=dtype)
    p = synth.make_inputs(cfg, seed=3, device=DEV, random_bias=True)
    fp = FewTokenPass(T, p["Wg"], p["W1"], p["b1"], p["W2"], p["b2"], k, 1)
    want = fp.forward(p["x"]).clone()
    streams = [torch.cuda.Stream() for _ in range(held)]
    for s in streams:                      # (and the sleeping kernel is loaded)
        with torch.cuda.stream(s):
            torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    first, last = event(), event()
    first.record()
    torch.cuda._sleep(CYCLES)
    last.record()
    torch.cuda.synchronize()
    length = first.elapsed_time(last)

    begin, done, ends = event(), event(), [event() for _ in streams]
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(CYCLES)
    torch.cuda._sleep(AHEAD)
    begin.record()
    got = fp.forward(p["x"])
    done.record()
    for s, e in zip(streams, ends):
        e.record(s)
    torch.cuda.synchronize()
    # held from before the call to after it
    assert all(begin.elapsed_time(e) < length for e in ends)
    assert all(done.elapsed_time(e) > 0 for e in ends)
    assert torch.equal(got, want) and int(fp.status.item()) == 0
