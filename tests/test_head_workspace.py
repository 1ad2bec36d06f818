"""The workspace that ``moe_head_workspace_size`` gives for a call with gradients also
holds the calls without them that an object made with gradients allows: scores, with
as many tokens or fewer (no GPU needed)."""
import random

import pytest

from mixture_experts_layer_11_gb300 import build as mbuild
from mixture_experts_layer_11_gb300 import ops


@pytest.fixture(scope="module", autouse=True)
def built():
    mbuild.build()


def size(T, V, d, dtype, piece=0, entries=1, grad=None):
    return ops.moe_head_workspace_size(ops.moe_head(T, piece, V, d, entries, dtype), grad)


def grad(dx=16, dW=16, dW_dtype=ops.MOE_F32):
    return ops.moe_head_grad(None, dx, dW, 1.0, 0, dW_dtype, 0)


CASES = [(4096, 1000, 2048, ops.MOE_BF16, 256), (32768, 131072, 4096, ops.MOE_BF16, 256),
         (65536, 32000, 2048, ops.MOE_BF16, 256), (32768, 32000, 768, ops.MOE_F32, 256),
         (131072, 32768, 65536, ops.MOE_BF16, 0), (600, 64, 4096, ops.MOE_F32, 1)]


@pytest.mark.parametrize("T,V,d,dtype,piece", CASES)
@pytest.mark.parametrize("g", [dict(), dict(dW=None), dict(dx=None), dict(dx=None, dW=None)], ids=str)
def test_workspace_with_gradients_holds_scores(T, V, d, dtype, piece, g):
    for wide in {ops.MOE_F32, dtype}:
        n = size(T, V, d, dtype, piece, grad=grad(dW_dtype=wide, **g))
        for t in (T, T // 2, 129, 128, 65, 64, 1):
            assert size(t, V, d, dtype, piece) <= n


def test_workspaces_over_many_shapes():
    rng = random.Random(3)

    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    for _ in range(4000):
        T, V, d, K = log(1, 1 << 18), log(1, 1 << 20), 8 * log(1, 2048), log(1, 128)
        dtype, piece = rng.choice([ops.MOE_F32, ops.MOE_BF16]), rng.choice([0, log(1, 1 << 17)])
        n = size(T, V, d, dtype, piece, K, grad(dW_dtype=rng.choice([ops.MOE_F32, dtype])))
        t, k = log(1, T), log(1, K)
        assert size(t, V, d, dtype, piece, k) <= n, (T, t, V, d, K, k, dtype, piece)
        assert size(t, V, d, dtype, 0, k) <= n
