"""check_status of the classes around the few-token layer and the gradient norm:
an error is raised once, and does not mark the calls after it."""
import pytest
import torch

from mixture_experts_layer_11_gb300 import build as mbuild
from mixture_experts_layer_11_gb300 import ops
from mixture_experts_layer_11_gb300.decode import FewTokenPass
from mixture_experts_layer_11_gb300.grads import GradClip


@pytest.fixture(scope="module", autouse=True)
def library():
    mbuild.build()


@pytest.mark.parametrize("kind", [FewTokenPass, GradClip])
@pytest.mark.parametrize("code", [ops.MOE_ERR_TIMEOUT, ops.MOE_ERR_NONFINITE])
def test_an_error_is_raised_once(kind, code):
    obj = object.__new__(kind)
    obj.status = torch.zeros(1, dtype=torch.int32)
    obj.check_status()
    obj.status.fill_(code)
    with pytest.raises(ops.MoEError) as e:
        obj.check_status()
    assert e.value.code == code
    obj.check_status()


@pytest.mark.gpu
def test_one_bad_step_does_not_mark_the_next():
    t = torch.ones(1000, device="cuda")
    c = GradClip([t])
    t[3] = float("nan")
    c.clip(1.0)
    with pytest.raises(ops.MoEError):
        c.check_status()
    t[3] = 1.0
    c.clip(1.0)
    c.check_status()
