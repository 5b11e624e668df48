"""The linear layer's path of few rows (5 to 16 of x at a small W), every number of
them, against 64 bits: x and W lie at the start of larger arrays of NaN, so a
value taken from a row that is not there would show."""
from __future__ import annotations

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import HALF_STEP, check, poisoned, rounded
from test_gpu_linear import BF, FP, fwd_bounds, inputs

pytestmark = pytest.mark.gpu
# 8 rows of W a workgroup, 16 with 16 waves, 16 with 4 waves; K: no whole piece of 64 values, some, a rest behind them
WIDTHS = [(8, 8), (8, 56), (64, 72), (136, 2040), (1032, 2056), (712, 16392)]


@pytest.mark.parametrize("n", range(5, 17))
def test_few_rows(gpu, n):
    for i, (k, m) in enumerate(WIDTHS):
        dt, act, bias, residual = (BF, FP)[(n + i) % 2], ("none", "silu", "gelu")[i % 3], i % 2 == 0, i > 3
        print(f"linear few rows n={n} k={k} m={m} {dt} {act} bias={bias} residual={residual}", flush=True)
        assert eg.engram_linear_fwd_workspace_bytes(n, k, m) == 0  # the path that takes none
        d = inputs(n, k, m, dt, gpu, seed=51)
        x, w = poisoned((n + 16, k), dt, gpu), poisoned((m + 16, k), dt, gpu)
        x[:n], w[:m] = d["x"], d["w"]
        _, _, y64, yerr = fwd_bounds(d, act, bias, residual)
        y = poisoned((n + 16, m), dt, gpu)
        eg.engram_linear_fwd(x[:n], w[:m], y[:n], bias=d["bias"] if bias else None,
                             residual=d["residual"] if residual else None, act=act)
        torch.cuda.synchronize()
        check("y", y[:n], y64, rounded(y64, dt) * (1 + 2 * HALF_STEP[dt]) + yerr * (1 + HALF_STEP[dt]))
        assert torch.isnan(y[n:]).all()
