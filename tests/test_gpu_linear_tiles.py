"""Every tile of the linear layer's products -- each shape with whole tiles, with
cut ones and with both, forward and both products of the backward, with every
kind of epilogue -- against 64 bits.  Each row says which tiles the plan gives
it as (shape, whole, cut, parts of a cut one), shapes in the order 256 x 256,
128 x 128, 128 x 128 of four stages, 64 x 128, 32 x 128; test_linear_plan_cpu.py
holds the plan to that."""
from __future__ import annotations

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import HALF_STEP, check, poisoned, rounded
from test_gpu_linear import BF, FP, buffer, bwd_bounds, fwd_bounds, inputs, run_bwd

pytestmark = pytest.mark.gpu

FORWARD = [  # n, k, m, tiles
    (3999, 5128, 5112, (0, 256, 64, 4)), (3245, 4744, 1416, (0, 0, 78, 3)), (1680, 272, 4632, (0, 133, 0, 1)),
    (3534, 792, 4744, (0, 256, 10, 3)), (520, 3640, 3272, (1, 0, 130, 3)), (3669, 968, 2192, (1, 512, 10, 4)),
    (101, 64, 168, (1, 2, 0, 1)), (87, 472, 80, (2, 0, 1, 2)), (463, 464, 152, (2, 8, 0, 1)),
    (791, 2280, 4616, (2, 256, 3, 9)), (51, 888, 64, (3, 0, 1, 3)), (58, 96, 88, (3, 1, 0, 1)),
    (34, 744, 98688, (3, 768, 3, 3)), (21, 744, 136, (4, 0, 2, 3)), (20, 88, 136, (4, 2, 0, 1)),
]
EPILOGUES = [("none", False, False, False), ("none", True, True, False), ("gelu", True, True, True),
             ("silu", False, False, False), ("none", False, False, True)]
BACKWARD = [  # n, k, m, tiles of grad_x, tiles of grad_w
    (445, 5552, 6952, (0, 0, 44, 5), (1, 2420, 0, 1)), (1905, 4440, 264, (0, 144, 0, 1), (2, 0, 105, 2)),
    (3227, 5296, 1040, (0, 256, 17, 4), (1, 378, 0, 1)), (139, 5416, 5424, (1, 0, 86, 5), (1, 1849, 0, 1)),
    (65, 8, 8, (1, 1, 0, 1), (4, 1, 0, 1)), (1852, 4384, 1144, (1, 512, 13, 4), (1, 315, 0, 1)),
    (66, 8, 456, (2, 0, 1, 2), (1, 4, 0, 1)), (799, 8, 464, (2, 7, 0, 1), (2, 0, 4, 3)),
    (791, 4632, 2416, (2, 256, 3, 8), (0, 190, 0, 1)), (33, 8, 760, (3, 0, 1, 3), (1, 6, 0, 1)),
    (33, 8, 8, (3, 1, 0, 1), (4, 1, 0, 1)), (2, 8, 712, (4, 0, 1, 3), (1, 6, 0, 1)),
    (724, 2560, 6608, (2, 0, 120, 2), (0, 256, 4, 3)), (3974, 264, 5488, (2, 0, 96, 2), (1, 0, 129, 3)),
    (1007, 4648, 1672, (1, 296, 0, 1), (1, 512, 6, 4)), (2244, 5424, 728, (0, 198, 0, 1), (2, 256, 2, 9)),
    (457, 8, 808, (2, 0, 4, 3), (2, 7, 0, 1)), (709, 8, 40, (1, 6, 0, 1), (3, 0, 1, 3)),
    (706, 8, 8, (1, 6, 0, 1), (4, 0, 1, 3)), (2, 8, 40, (4, 1, 0, 1), (3, 1, 0, 1)),
    (6952, 5552, 448, (1, 2420, 0, 1), (0, 0, 44, 5)),
]


@pytest.mark.parametrize("n,k,m,tiles", FORWARD)
def test_forward(gpu, n, k, m, tiles):
    for i, (act, bias, residual, z) in enumerate(EPILOGUES):
        dt = (BF, FP)[i % 2]
        print(f"linear tiles fwd n={n} k={k} m={m} {dt} {act} bias={bias} residual={residual} z={z}", flush=True)
        d = inputs(n, k, m, dt, gpu, seed=41)
        z64, zerr, y64, yerr = fwd_bounds(d, act, bias, residual)
        y, zo = poisoned((n, m), dt, gpu), poisoned((n, m), dt, gpu)
        eg.engram_linear_fwd(d["x"], d["w"], y, buffer(eg.engram_linear_fwd_workspace_bytes(n, k, m), gpu),
                             bias=d["bias"] if bias else None, residual=d["residual"] if residual else None,
                             z=zo if z else None, act=act)
        torch.cuda.synchronize()
        check("y", y, y64, rounded(y64, dt) * (1 + 2 * HALF_STEP[dt]) + yerr * (1 + HALF_STEP[dt]))
        if z:
            check("z", zo, z64, rounded(z64, dt) + 2 * zerr)


@pytest.mark.parametrize("n,k,m,dx,dw", BACKWARD)
def test_backward(gpu, n, k, m, dx, dw):
    for dt, act in ((BF, "none"), (FP, "gelu")):
        print(f"linear tiles bwd n={n} k={k} m={m} {dt} {act}", flush=True)
        d = inputs(n, k, m, dt, gpu, seed=42)
        bounds = bwd_bounds(d, act)
        out = poisoned((n, k), dt, gpu), poisoned((m, k), dt, gpu), poisoned((m,), torch.float32, gpu)
        run_bwd(d, d["x"], d["grad_y"], act, *out)
        torch.cuda.synchronize()
        for name, got, bound in zip(("grad_x", "grad_w", "grad_bias"), out, bounds):
            check(name, got, *bound)
