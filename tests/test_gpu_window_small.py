"""The window attention in half precision where numbers are small: gradients of
ordinary small size over many keys.  What is rounded to fp16 as an operand has to
keep fp16's digits there, not its smallest step."""
from __future__ import annotations

import math

import pytest
import torch

from layers_util import F32, HALF_STEP
from test_gpu_window_attn import case, run_backward, run_forward, visible

pytestmark = pytest.mark.gpu
FP = torch.float16
U, LEAST = HALF_STEP[FP], 2.0 ** -25  # half a step of fp16, relative and (below 2^-14) absolute


def gradients(c, o, lse):
    """Exact gradients, and for each the size of its error if every rounding were independent: the operands' (half
    a step, at most 2^-29 of the largest d of its sum, 2^-39 for a weight), the output's, and, as they are common to a row,
    what the given o and lse are off by, added up as absolute values."""
    out = []
    q, k, v, g = (c[x].double() for x in ("q", "k", "v", "go"))
    n, per = c["n"], c["hq"] // c["hk"]
    seen = visible(n, c["window"], c["sinks"]).to(q.device)
    totals = [torch.zeros_like(x) for x in (q, k, v)]
    squares = [torch.zeros_like(x) for x in (q, k, v)]
    common = [torch.zeros_like(x) for x in (q, k, v)]
    for h in range(c["hq"]):
        kh = h // per
        z = (c["scale"] * (q[:, h] @ k[:, kh].t())).masked_fill(~seen, -math.inf)
        p, ls = torch.softmax(z, 1), torch.logsumexp(z, 1)
        o64 = p @ v[:, kh]
        dp, delta = g[:, h] @ v[:, kh].t(), (g[:, h] * o64).sum(1, keepdim=True)
        d = p * (dp - delta)
        # scores in fp32 and the given lse: relative to a weight
        off = (lse[:, h].double() - ls).abs()[:, None] + F32 * (c["d"] + 8) * (2 + z.masked_fill(~seen, 0).abs())
        shift = (g[:, h] * (o[:, h].double() - o64)).sum(1, keepdim=True).abs() + \
            F32 * (c["d"] + 8) * (g[:, h].abs() * o64.abs()).sum(1, keepdim=True)
        ed = p * shift + off * d.abs()
        totals[0][:, h] = c["scale"] * (d @ k[:, kh])
        totals[1][:, kh] += c["scale"] * (d.t() @ q[:, h])
        totals[2][:, kh] += p.t() @ g[:, h]
        row = (U * d) ** 2 + (2.0 ** -29 * d.abs().amax(1, keepdim=True) * seen) ** 2
        column = (U * d) ** 2 + (2.0 ** -29 * d.abs().amax(0, keepdim=True) * seen) ** 2
        squares[0][:, h] = c["scale"] ** 2 * (row @ k[:, kh] ** 2)
        squares[1][:, kh] += c["scale"] ** 2 * (column.t() @ q[:, h] ** 2)
        squares[2][:, kh] += ((U * p) ** 2 + (2.0 ** -39 * seen) ** 2).t() @ g[:, h] ** 2
        common[0][:, h] = c["scale"] * (ed @ k[:, kh].abs())
        common[1][:, kh] += c["scale"] * (ed.t() @ q[:, h].abs())
        common[2][:, kh] += (off * p).t() @ g[:, h].abs()
    for t, s, e in zip(totals, squares, common):
        out.append((t, torch.sqrt(s + (U * t.abs() + LEAST) ** 2), e))
    return out


def check_norms(c, dev, dims, names=("grad_q", "grad_k", "grad_v")):
    """Norms of the errors over `dims`: roundings are even over their half step, so their norm is below that of the
    half steps by a third of its square; the common errors at their worst, all of one sign, add a norm of their own, of
    which a row's products take a share like its rounding's."""
    o, lse = run_forward(c, dev)
    for name, got, (want, rounding, common) in zip(("grad_q", "grad_k", "grad_v"), run_backward(c, o, lse, dev),
                                                   gradients(c, o, lse)):
        if name not in names:
            continue
        off = (got.double() - want).square().sum(dims).sqrt()
        bound = rounding.square().sum(dims).sqrt() + common.square().sum(dims).sqrt()
        at = (off / bound).max().item()
        print(f"{name}: {at:.2f} of the bound, off by {(off / want.square().sum(dims).sqrt()).max().item():.2e}", flush=True)
        assert at <= 1, name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("window,sinks", [(1 << 40, 0), (1500, 7)])
def test_gradients_of_every_size(gpu, window, sinks, size, d):
    c = case([3000], 2, 1, d, FP, gpu, window, sinks, seed=d, std=1.0)
    c["go"] = (c["go"].float() * size).to(FP)
    check_norms(c, gpu, (0, 1, 2))


def test_gradients_whose_size_grows_along_the_sequence(gpu):
    """Each row's and each key's gradient by itself, sizes from 2^-13 to 2^12 in one sequence, in both directions."""
    n = 1024
    for way in (1, -1):
        c = case([n], 4, 2, 128, FP, gpu, 1 << 40, 0, seed=3, std=1.0)
        grow = torch.linspace(-13 * way, 12 * way, n, device=gpu)[:, None, None]
        c["go"] = (c["go"].float() * torch.exp2(grow)).to(FP)
        check_norms(c, gpu, 2)
