"""The activations of the linear layer and their slopes where they are small, held
relative to themselves: z comes in through the bias (a matrix of zeros before
it), the slope goes out through grad_bias in fp32."""
from __future__ import annotations

import math

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import HALF_STEP, TINY, check, poisoned
from test_gpu_linear import BF, FP, buffer

pytestmark = pytest.mark.gpu
# An exponential of x is off by 2^-23 of |x| (its argument's two roundings) and two steps; |x| is below 104, and a
# power that small is below the smallest normal value: 2^-16 + 2^-22.  The normal distribution's tail adds 2e-7 and
# a dozen fp32 operations, the products and sums after it a few 2^-24.
REL = 2.0 ** -15
NORMAL = 2.0 ** -126  # below it a value may be zero


def silu(z):
    return z * torch.sigmoid(z), torch.sigmoid(z), z * torch.sigmoid(z) * torch.sigmoid(-z)


def gelu(z):
    cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
    return z * cdf, cdf, z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


ACTS = {"silu": (silu, 104.0), "gelu": (gelu, 14.5)}


def points(act, dev):
    """A multiple of 8 values of z: dense where the result is small, and the other side."""
    far = ACTS[act][1]
    return torch.cat((torch.linspace(-far, 0, 4096), torch.linspace(-12, 12, 4088),
                      torch.tensor([-30.0, -1e4, -1e30, 30.0, 100.0, 1e30, -0.0, 1e-30]))).to(dev)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("n", [1, 9, 70])  # rows of W, few rows, tiles
def test_values(gpu, act, dt, n):
    z = points(act, gpu)
    if dt == FP:
        z = z.clamp(-6e4, 6e4)
    m = z.numel()
    x, w = torch.zeros((n, 8), dtype=dt, device=gpu), torch.zeros((m, 8), dtype=dt, device=gpu)
    y = poisoned((n, m), dt, gpu)
    eg.engram_linear_fwd(x, w, y, buffer(eg.engram_linear_fwd_workspace_bytes(n, 8, m), gpu), bias=z, act=act)
    torch.cuda.synchronize()
    want = ACTS[act][0](z.double())[0]
    err = REL * want.abs() + NORMAL * (1 + z.double().abs().clamp(max=128))
    check(act, y, want.expand(n, m), ((1 + HALF_STEP[dt]) * err + HALF_STEP[dt] * want.abs() + TINY[dt]).expand(n, m))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [BF, FP])
def test_slopes(gpu, act, dt):
    z = points(act, gpu)
    if dt == FP:
        z = z.clamp(-6e4, 6e4)
    z = z.to(dt)[None]
    m = z.numel()
    x, w = torch.zeros((1, 8), dtype=dt, device=gpu), torch.zeros((m, 8), dtype=dt, device=gpu)
    gb = poisoned((m,), torch.float32, gpu)
    eg.engram_linear_bwd(torch.ones((1, m), dtype=dt, device=gpu), x, w, None, None,
                         buffer(eg.engram_linear_bwd_workspace_bytes(1, 8, m), gpu), z=z, grad_bias=gb, act=act)
    torch.cuda.synchronize()
    _, p, rest = ACTS[act][0](z[0].double())  # the slope is the sum of two terms, of opposite signs below 0
    check(act, gb, p + rest, REL * (p + rest.abs()) + NORMAL * (1 + z[0].double().abs().clamp(max=128)))


@pytest.mark.parametrize("dt", [BF, FP])
def test_range_of_the_activations_gradient(gpu, dt):
    """The products take grad_y act'(z) in the element type: within bf16's range wherever grad_y is, in
    fp16 infinite above 65504 and in whole steps of 2^-24 below 2^-14; grad_bias takes it in fp32."""
    z = torch.tensor([[1.5, -1.5, 0.0, 1.5, -5.0, 0.5, 3.0, 30.0]], device=gpu).to(dt)
    gy = torch.tensor([[65000.0, 65000.0, 65000.0, -65000.0, 2.0 ** -12, 2.0 ** -24, 2.0 ** -20, 65504.0]], device=gpu).to(dt)
    w = torch.eye(8, device=gpu).to(dt)
    x = torch.ones((1, 8), dtype=dt, device=gpu)
    gw, gb = poisoned((8, 8), dt, gpu), poisoned((8,), torch.float32, gpu)
    eg.engram_linear_bwd(gy, x, w, None, gw, buffer(eg.engram_linear_bwd_workspace_bytes(1, 8, 8), gpu), z=z, grad_bias=gb,
                         act="gelu")
    torch.cuda.synchronize()
    _, p, rest = gelu(z[0].double())
    dz = gy[0].double() * (p + rest)
    check("grad_bias", gb, dz, REL * gy[0].double().abs() * (p + rest.abs()))
    kept = dz.to(dt).double()
    assert torch.isinf(kept).tolist() == [dt == FP, False, False, dt == FP, False, False, False, False]
    # rounded here and, a little off by REL, there: a step apart at most
    step = 2 * HALF_STEP[dt] * kept.abs().nan_to_num(0, 0, 0) + TINY[dt]
    check("grad_w", gw, kept[:, None].expand(8, 8), step[:, None].expand(8, 8))
