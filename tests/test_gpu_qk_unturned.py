"""Values that the rotation does not reach (from R on, or all of them at R = 0):
what is not finite in one of them stays in it, forward and backward."""
from __future__ import annotations

import math

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import F32, check, poisoned, rounded
from test_gpu_qk_norm_rope import ANGLE, BF, EPS, F4, FP, backward64, case, factors, forward64, partner_abs, run_bwd

pytestmark = pytest.mark.gpu
CASES = [(64, 32, False, BF), (64, 32, True, FP), (128, 0, False, F4), (40, 16, False, F4), (24, 16, True, BF)]


@pytest.mark.parametrize("d,r,inter,dt", CASES)
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_forward(gpu, d, r, inter, dt, bad):
    """An infinite value: its root mean square is infinite too, so the others become 0 and it NaN.  An
    infinite weight: its value is infinite and the others are what they were."""
    c = case(3, 4, 2, d, r, dt, gpu, seed=31)
    cos, sin = factors(c["positions"], r) if r else (None, None)
    c["q"][1, 2, r + 5] = bad
    c["wk"][r + 6] = bad
    qo, ko = poisoned((3, 4, d), dt, gpu), poisoned((3, 2, d), dt, gpu)
    eg.engram_qk_norm_rope_fwd(c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["freqs"], qo, ko, eps=EPS,
                               interleaved=inter)
    torch.cuda.synchronize()
    for name, x, w, got in (("q_out", c["q"], c["wq"], qo), ("k_out", c["k"], c["wk"], ko)):
        want = forward64(x.double(), w.double(), cos, sin, r, inter)
        size = partner_abs(forward64(x.double(), w.double(), None, None, 0, inter), r, inter)
        check(name, got, want, rounded(want, dt) + 2 * (F32 * (d + 8) + ANGLE[dt]) * size)


@pytest.mark.parametrize("d,r,inter,dt", CASES)
@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_backward(gpu, d, r, inter, dt, bad):
    """An infinite gradient of one value: the head's gradients are not finite, the weights' gradients of
    the other columns are what they were, bit for bit."""
    c = case(3, 4, 2, d, r, dt, gpu, seed=32)
    clean = run_bwd(c, inter, dt, gpu)
    c["gq"][1, 2, r + 5] = bad
    gq, gk, gwq, gwk = run_bwd(c, inter, dt, gpu)
    cos, sin = factors(c["positions"], r) if r else (None, None)
    want = backward64(c["gq"].double(), c["q"].double(), c["wq"].double(), cos, sin, r, inter)
    assert torch.equal(torch.isfinite(gwq), torch.isfinite(want[1]))
    keep = torch.arange(d, device=gpu) != r + 5
    assert torch.equal(gwq[keep], clean[2][keep]) and gwq[r + 5] == want[1][r + 5]
    assert torch.equal(gk.view(torch.uint8), clean[1].view(torch.uint8)) and torch.equal(gwk, clean[3])
    rows = torch.ones((3, 4), dtype=torch.bool, device=gpu)
    rows[1, 2] = False
    assert torch.equal(gq[rows].view(torch.uint8), clean[0][rows].view(torch.uint8))
    assert not torch.isfinite(gq[1, 2]).any()
