"""The window attention in half precision where numbers are small: gradients of
ordinary small size over many keys, keys whose weights lie near the bottom of
fp16's range, and very many keys beside one that has nearly all of the weight.
What is rounded to fp16 as an operand has to keep fp16's digits there, not its
smallest step."""
from __future__ import annotations

import math

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import F32, HALF_STEP, poisoned
from test_gpu_window_attn import case, run_backward, run_forward, visible

pytestmark = pytest.mark.gpu
FP, F4 = torch.float16, torch.float32
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


def test_weights_at_the_bottom_of_the_range(gpu):
    """Keys of weights down to 2^-24 for all of their rows: each key's own gradients keep their digits."""
    n = 512
    c = case([n], 2, 1, 64, FP, gpu, 1 << 40, 0, seed=4, std=0.0)
    c["q"][:, :, 0] = 4.0
    c["k"][:, :, 0] = (-torch.linspace(0, 24, n, device=gpu) * math.log(2) / (4.0 * c["scale"])).to(FP)[:, None]
    c["go"] = (c["go"].float() * 200.0).to(FP)
    check_norms(c, gpu, 2, names=("grad_v",))


def beside_one(n, dev):
    """Values behind the first token have a weight of 2^-25.5 of the first's each."""
    g = torch.Generator().manual_seed(5)
    d = 64
    q, k = torch.zeros((n, 1, d)), torch.zeros((n, 1, d))
    q[..., 0] = 4.0
    k[1:, :, 0] = -25.5 * math.log(2) / 4.0 + 0.01 * torch.randn((n - 1, 1), generator=g)
    v = 1.0 + 0.25 * torch.randn((n, 1, d), generator=g)
    v[0] = 0.0
    return [x.to(FP).to(dev) for x in (q, k, v)]


def last_row(q, k, v):
    p = torch.softmax((q[-1, 0].double() * k[:, 0].double()).sum(1), 0)
    o = p @ v[:, 0].double()
    # a weight's rounding to fp16, at most 2^-32 of the largest; its exponent in fp32; the sums; the output
    bound = p @ v[:, 0].double().abs() * (U + F32 * 64) + 2.0 ** -32 * p.max() * v[:, 0].double().abs().sum(0) + U * o.abs() + LEAST
    return o, bound


def test_very_many_keys_beside_a_peak(gpu):
    n = 100001
    q, k, v = beside_one(n, gpu)
    o, lse = poisoned((n, 1, 64), FP, gpu), poisoned((n, 1), F4, gpu)
    eg.engram_window_attn_fwd(q, k, v, torch.tensor([0, n], device=gpu), o, 1 << 40, lse=lse, scale=1.0)
    want, bound = last_row(q, k, v)
    print(o[-1, 0, :3].tolist(), want[:3].tolist(), flush=True)
    assert ((o[-1, 0].double() - want).abs() <= bound).all()
    ls = torch.logsumexp((q[-1, 0].double() * k[:, 0].double()).sum(1), 0)
    # one lane after the other adds half of the terms, each sum rounded: n / 2 times 2^-24 of it (terms of 2^-25.5 beside
    # 1 are all lost in the lane that has the 1); then log2 and its two roundings
    assert abs(lse[-1, 0].double() - ls) <= F32 * (n / 2 + 64)


def test_single_tokens_over_many_lines(gpu):
    """As many heads as fill the chip, so that lists are not split: a wave has a quarter of one, the first one's the peak."""
    n, heads = 20001, 512
    _, k, v = beside_one(n, gpu)
    k, v = k[:, :, :8], v[:, :, :8]
    q = torch.zeros((1, heads, 8), dtype=FP, device=gpu)
    q[..., 0] = 4.0
    ck, cv = (torch.empty((1, heads, n, 8), dtype=FP, device=gpu) for _ in range(2))
    ck[0], cv[0] = k[:, 0], v[:, 0]
    ck[0, :, -1], cv[0, :, -1] = math.nan, math.nan  # the token's own line
    assert eg.engram_window_attn_step_workspace_bytes(1, heads, heads, 8, n) == 0
    o = poisoned((1, heads, 8), FP, gpu)
    own = [x[-1:].expand(1, heads, 8).contiguous() for x in (k, v)]
    eg.engram_window_attn_step(q, *own, ck, cv, torch.tensor([0], device=gpu), torch.tensor([n - 1], device=gpu), o, None, n,
                               scale=1.0)
    want, bound = last_row(q[:, :1], k, v)
    print(o[0, 0, :3].tolist(), want[:3].tolist(), flush=True)
    assert ((o[0].double() - want).abs() <= bound).all()
