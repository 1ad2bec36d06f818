"""The losses over a vocabulary head refuse bad arguments on the host, before
anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_11_gb300 import build as mbuild
from mixture_experts_layer_11_gb300 import ops


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return ops.lib()


def _head(T=5, V=1000, d=256, dtype=ops.MOE_BF16, entries=1, piece=0):
    return ops.moe_head(T, piece, V, d, entries, dtype)


def _grad(weight=None, dx=16, dW=16, scale=1.0, mean=0, dW_dtype=ops.MOE_BF16, accumulate=0):
    return ops.moe_head_grad(weight, dx, dW, scale, mean, dW_dtype, accumulate)


def _ce(lib, h, g=None, x=16, W=16, target=16, loss=16, lse=16, ws=16, status=16):
    return lib.moe_head_ce(ctypes.byref(h), x, W, target, loss, lse,
                           None if g is None else ctypes.byref(g), ws, status, None)


def _distill(lib, h, g=None, x=16, W=16, idx=16, logits=16, temperature=1.0, loss=16, lse=16,
             ws=16, status=16):
    return lib.moe_head_distill(ctypes.byref(h), x, W, idx, logits, temperature, loss, lse,
                                None if g is None else ctypes.byref(g), ws, status, None)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(V=0), dict(d=0), dict(dtype=7), dict(entries=0),
                                 dict(piece=-1)])
def test_refuses_invalid_shapes(lib, bad):
    h = _head(**bad)
    assert _ce(lib, h) == ops.MOE_ERR_INVALID
    assert _distill(lib, h, _grad()) == ops.MOE_ERR_INVALID
    assert ops.moe_head_workspace_size(h) == 0


@pytest.mark.parametrize("bad", [dict(T=(1 << 30) + 1), dict(V=(1 << 22) + 1), dict(d=12), dict(d=(1 << 20) + 8),
                                 dict(entries=129), dict(piece=(1 << 30) + 1)])
def test_refuses_unsupported_shapes(lib, bad):
    h = _head(**bad)
    assert _distill(lib, h) == ops.MOE_ERR_UNSUPPORTED
    assert ops.moe_head_workspace_size(h, _grad()) == 0


@pytest.mark.parametrize("bad", [dict(x=None), dict(W=None), dict(target=None), dict(loss=None), dict(ws=None),
                                 dict(x=8), dict(W=24), dict(target=20), dict(loss=18), dict(lse=18),
                                 dict(ws=8), dict(status=2)])
def test_refuses_bad_pointers(lib, bad):
    assert _ce(lib, _head(), **bad) == ops.MOE_ERR_INVALID
    if "target" in bad:
        bad = dict(idx=bad["target"])
    assert _distill(lib, _head(entries=4), _grad(), **bad) == ops.MOE_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(logits=None), dict(logits=18), dict(temperature=0.0), dict(temperature=-1.0),
                                 dict(temperature=float("nan")), dict(temperature=float("inf")),
                                 dict(temperature=9e-5), dict(temperature=1.1e4)])
def test_distill_refuses(lib, bad):
    assert _distill(lib, _head(entries=4), **bad) == ops.MOE_ERR_INVALID


@pytest.mark.parametrize("bad,code", [
    (dict(mean=2), ops.MOE_ERR_INVALID), (dict(accumulate=2), ops.MOE_ERR_INVALID),
    (dict(dW_dtype=5), ops.MOE_ERR_INVALID), (dict(dx=8), ops.MOE_ERR_INVALID),
    (dict(dW=8), ops.MOE_ERR_INVALID), (dict(weight=18), ops.MOE_ERR_INVALID),
    (dict(accumulate=1), ops.MOE_ERR_UNSUPPORTED)])
def test_refuses_bad_gradients(lib, bad, code):
    assert _ce(lib, _head(), _grad(**bad)) == code
    assert _distill(lib, _head(entries=4), _grad(**bad)) == code


def test_refuses_bf16_gradient_of_an_fp32_head(lib):
    assert _ce(lib, _head(dtype=ops.MOE_F32), _grad()) == ops.MOE_ERR_INVALID


def test_cross_entropy_takes_one_target(lib):
    assert _ce(lib, _head(entries=2)) == ops.MOE_ERR_INVALID
    assert lib.moe_head_ce(None, 16, 16, 16, 16, 16, None, 16, 16, None) == ops.MOE_ERR_INVALID


def test_without_tokens_does_nothing(lib):
    h = _head(T=0)
    assert _ce(lib, h, x=None, W=None, target=None, loss=None, lse=None, ws=None) == ops.MOE_OK
    assert _ce(lib, h, _grad(dW=None, dx=None), x=None, target=None, loss=None, ws=None) == ops.MOE_OK


@pytest.mark.parametrize("grad", [None, dict(), dict(dW_dtype=ops.MOE_F32)])
@pytest.mark.parametrize("kw", [dict(), dict(V=50257), dict(piece=512), dict(entries=128), dict(d=8, V=1)])
def test_workspace_of_more_tokens_holds_fewer(lib, kw, grad):
    g = None if grad is None else _grad(**grad)
    sizes = [ops.moe_head_workspace_size(_head(T=t, **kw), g) for t in (0, 1, 127, 128, 129, 511, 512, 513, 5000)]
    assert sizes[0] > 0 and sizes == sorted(sizes)


def test_workspace_is_bounded(lib):
    # what is held a logit stays within 2 GiB, whatever the tokens
    a, b = (ops.moe_head_workspace_size(_head(T=t, V=131072, d=64), _grad(dW_dtype=ops.MOE_F32))
            for t in (1 << 15, 1 << 17))
    assert a < 2.2 * 2 ** 30 and b - a <= (1 << 17) * (64 * 2 + 64)


def test_binding_refuses():
    from mixture_experts_layer_11_gb300.head import HeadLoss
    W = torch.zeros(100, 64)
    for bad in (dict(W=W[0]), dict(W=W.half()), dict(T=-1), dict(piece=-1), dict(entries=0),
                dict(entries=129), dict(dW=W, backward=False), dict(dW=W, want_dW=False),
                dict(dW=W[:50]), dict(dW=W.double())):
        args = dict(T=5, W=W)
        args.update(bad)
        with pytest.raises(ValueError):
            HeadLoss(args.pop("T"), args.pop("W"), **args)
    with pytest.raises(ops.MoEError):
        HeadLoss(5, W)                                  # not on a CUDA device


def test_reference_in_64_bits():
    """The formulas that the kernels are held to, against automatic differentiation."""
    from head_util import make, make_entries, reference
    x, W, target = make(12, 16, 40, torch.float64, device="cpu")
    idx, logits = make_entries(12, 5, 40, target, device="cpu")
    idx[3] = -1
    target[3] = -1
    idx[4, 2:] = -1
    weight = torch.rand(12, dtype=torch.float64)
    live = target >= 0
    for tau, kind in ((1.0, "ce"), (1.7, "distill")):
        a, b = x.clone().requires_grad_(), W.clone().requires_grad_()
        z = a @ b.T / tau
        if kind == "ce":
            loss = torch.nn.functional.cross_entropy(z, target, ignore_index=-1, reduction="none")
            got, _ = reference(x, W, target=target, weight=weight, scale=0.3, mean=True)
        else:
            t = (logits.double() / tau).masked_fill(idx < 0, float("-inf"))
            q = torch.where(live[:, None], torch.softmax(t, 1), 0.0)
            logp = torch.log_softmax(z, 1).gather(1, idx.clamp(min=0))
            loss = tau ** 2 * torch.where(q > 0, q * (torch.log(q.clamp(min=1e-300)) - logp), 0.0).sum(1)
            got, _ = reference(x, W, idx=idx, logits=logits, temperature=tau, weight=weight, scale=0.3,
                               mean=True)
        (0.3 * (loss * weight)[live].sum() / live.sum()).backward()
        for u, v in ((got["loss"], loss.detach()), (got["dx"], a.grad), (got["dW"], b.grad)):
            assert (u - v).abs().max() <= 1e-12
