"""The entry points for a few tokens and for gradient norms refuse bad
arguments on the host, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_11_gb300 import build as mbuild
from mixture_experts_layer_11_gb300 import ops


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return ops.lib()


def _shape(**kw):
    base = dict(T=5, d=256, f=512, E=8, k=2, dtype="bf16", renorm=1)
    base.update(kw)
    return ops.make_shape(**base)


def _few(lib, s, x=16, residual=None, y=16, ws=16, status=16, **params):
    p = dict(Wg=16, logit_bias=None, W1=16, b1=None, W2=16, b2=None)
    p.update(params)
    return lib.moe_layer_few(ctypes.byref(s), ctypes.byref(ops.moe_layer_params(**p)), x, residual,
                             y, ws, status, None)


@pytest.mark.parametrize("bad", [dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(T=-1),
                                 dict(d=0), dict(dtype=7), dict(renorm=2)])
def test_few_refuses_invalid_shapes(lib, bad):
    assert _few(lib, _shape(**bad)) == ops.MOE_ERR_INVALID
    assert ops.moe_layer_few_workspace_size(_shape(**bad)) == 0


@pytest.mark.parametrize("bad", [dict(T=65), dict(d=12), dict(f=12), dict(d=260, dtype="f32"),
                                 dict(T=64, E=256, k=16, d=1 << 17, f=1 << 17, dtype="f32")])
def test_few_refuses_unsupported_shapes(lib, bad):
    assert _few(lib, _shape(**bad)) == ops.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(x=None), dict(y=None), dict(ws=None), dict(x=8), dict(y=24),
                                 dict(residual=8), dict(ws=8), dict(status=2), dict(Wg=None),
                                 dict(W1=None), dict(W2=None), dict(b1=8), dict(b2=8), dict(W2=8),
                                 dict(logit_bias=8)])
def test_few_refuses_bad_pointers(lib, bad):
    assert _few(lib, _shape(), **bad) == ops.MOE_ERR_INVALID


def test_few_refuses_no_parameters(lib):
    s = _shape()
    assert lib.moe_layer_few(ctypes.byref(s), None, 16, None, 16, 16, 16, None) == ops.MOE_ERR_INVALID
    assert lib.moe_layer_few(None, None, 16, None, 16, 16, 16, None) == ops.MOE_ERR_INVALID


def test_few_without_tokens_does_nothing(lib):
    assert _few(lib, _shape(T=0), x=None, y=None, ws=None) == ops.MOE_OK


def test_few_workspace_size(lib):
    assert ops.moe_layer_few_workspace_size(_shape(T=64)) > 0
    assert ops.moe_layer_few_workspace_size(_shape(T=65)) == 0
    # a call with fewer tokens fits the workspace of one with more
    for kw in (dict(), dict(E=1, k=1), dict(E=128, k=8, d=4096, f=1024), dict(dtype="f32"),
               dict(d=768, f=3072), dict(d=8, f=8)):
        sizes = [ops.moe_layer_few_workspace_size(_shape(T=t, **kw)) for t in range(1, 65)]
        assert sizes == sorted(sizes)


def _grads(*g):
    return (ops.moe_grad * len(g))(*[ops.moe_grad(*x) for x in g])


@pytest.mark.parametrize("fn", ["norm", "clip"])
@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(g=None), dict(norm=None), dict(norm=18), dict(ws=None), dict(ws=8),
    dict(status=2), dict(g=[(None, None, 3, 0)]), dict(g=[(18, None, 3, 0)]), dict(g=[(17, None, 3, 1)]),
    dict(g=[(16, 18, 3, 0)]), dict(g=[(16, 17, 3, 1)]), dict(g=[(16, None, -1, 0)]),
    dict(g=[(16, None, 3, 2)])])
def test_grads_refuse_bad_arguments(lib, fn, bad):
    a = dict(n=1, g=[(16, None, 3, 0)], norm=16, ws=16, status=16)
    a.update(bad)
    g = None if a["g"] is None else _grads(*a["g"])
    if fn == "norm":
        code = lib.moe_grad_norm(a["n"], g, a["norm"], a["ws"], a["status"], None)
    else:
        code = lib.moe_grad_clip(a["n"], g, 1.0, a["norm"], a["ws"], a["status"], None)
    assert code == ops.MOE_ERR_INVALID


def test_grads_refuse_more_than_any_memory(lib):
    g = _grads((16, None, 1 << 44, 0))
    assert lib.moe_grad_norm(1, g, 16, 16, 16, None) == ops.MOE_ERR_UNSUPPORTED
    g = _grads(*[(16, None, 1 << 42, 0)] * 3)
    assert lib.moe_grad_norm(3, g, 16, 16, 16, None) == ops.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("bound", [-1.0, float("nan"), -float("inf")])
def test_clip_refuses_bad_bounds(lib, bound):
    assert lib.moe_grad_clip(1, _grads((16, None, 3, 0)), bound, 16, 16, 16, None) == ops.MOE_ERR_INVALID


def test_grads_workspace_size(lib):
    assert ops.moe_grad_workspace_size(-1) == 0
    sizes = [ops.moe_grad_workspace_size(n) for n in (0, 1, 100, 1000, 10000)]
    assert sizes[0] > 0 and sizes == sorted(sizes)


def test_bindings_refuse_tensors_the_library_cannot_check():
    t = torch.zeros(4)
    with pytest.raises(ops.MoEError):
        ops.make_grads([t])                       # not on a CUDA device
    with pytest.raises(ops.MoEError):
        ops.make_grads([t.half()])                # type
    with pytest.raises(ops.MoEError):
        ops.make_grads([t], [t, t])               # another number of outs
    with pytest.raises(ops.MoEError):
        ops.make_layer_params(_shape(dtype="f32"), t, None, t, None, t, None)
    from mixture_experts_layer_11_gb300.decode import FewTokenPass
    W1, W2, Wg = torch.zeros(2, 16, 8), torch.zeros(2, 8, 16), torch.zeros(2, 8)
    with pytest.raises(ValueError):
        FewTokenPass(65, Wg, W1, None, W2, None, 1, 0)
    with pytest.raises(ValueError):
        FewTokenPass(1, Wg[:1], W1, None, W2, None, 1, 0)
    with pytest.raises(ValueError):
        FewTokenPass(1, Wg.half(), W1.half(), None, W2.half(), None, 1, 0)
