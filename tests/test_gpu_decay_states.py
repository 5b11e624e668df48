"""The decay attention's states, which the caller gets in fp32: what a state keeps
of its past under every decay, held relative to that itself (no larger terms
beside it that would hide it), and infinite states."""
from __future__ import annotations

import math

import pytest
import torch

from layers_util import F32, check
from test_gpu_decay_attn import case, recurrence, reversed_recurrence, run_bwd, run_fwd

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
RATES = [0.0, -1e-6, -0.002, -0.01, -0.05, -0.2, -0.5, -1.0, -math.inf]


def kept(c):
    """lam^length for each sequence and head, and its relative error: the exponent |log lam| length is a
    product of three fp32 values (the logarithm to base 2, a constant's rounding and the steps), each step of
    64 rows is an exponential (two steps of fp32) and two roundings, a border between segments as much again."""
    ld = c["ld"].double().cpu()
    t = torch.tensor(c["lens"], dtype=torch.float64)[:, None]
    x = torch.where(t == 0, torch.zeros_like(t), torch.nan_to_num(ld, neginf=-1e300)[None] * t)
    chunks = 2 * (t / 64 + 2)
    return torch.exp(x)[..., None, None], F32 * (4 * torch.where(x < -1e3, 0 * x, -x) + 4 * chunks)[..., None, None]


@pytest.mark.parametrize("lens", [[1], [64], [63, 0, 65], [200], [700, 130]])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 40)])
def test_a_state_that_only_decays(gpu, lens, dk, dv):
    """Keys (backward: queries) of zeros add nothing, so the last state is the first one's share; below
    2^-126, the smallest normal value, a power may be zero."""
    print(f"decay states lens={lens} dk={dk} dv={dv}", flush=True)
    c = case(lens, len(RATES), dk, dv, gpu, True, ld=torch.tensor(RATES), seed=21)
    c["k"].zero_()
    _, out = run_fwd(c, gpu)
    share, err = kept(c)
    s0 = c["s0"].double().cpu()
    check("state_out", out, (share * s0).to(gpu), (err * share * s0.abs() + 2.0 ** -126 * s0.abs()).to(gpu))
    c["q"].zero_()
    gin = run_bwd(c, gpu)[3]
    ds = c["ds"].double().cpu()
    check("grad_state_in", gin, (share * ds).to(gpu), (err * share * ds.abs() + 2.0 ** -126 * ds.abs()).to(gpu))


@pytest.mark.parametrize("lens", [[40], [150, 90], [400]])
def test_infinite_states(gpu, lens):
    """An infinity in a carried state stays one, of its sign, and no other entry changes."""
    c = case(lens, 2, 64, 64, gpu, True, ld=torch.tensor([-0.01, -0.4]), seed=22)
    _, clean = run_fwd(c, gpu)
    clean_in = run_bwd(c, gpu)[3]
    c["s0"][0, 1, 3, 5], c["s0"][0, 0, 7, 9] = math.inf, -math.inf
    c["ds"][0, 1, 3, 5], c["ds"][0, 0, 7, 9] = math.inf, -math.inf
    _, out = run_fwd(c, gpu)
    gin = run_bwd(c, gpu)[3]
    for got, want in ((out, clean), (gin, clean_in)):
        want[0, 1, 3, 5], want[0, 0, 7, 9] = math.inf, -math.inf
        assert torch.equal(got, want), (got != want).nonzero()


@pytest.mark.parametrize("what", ["k", "v", "q", "do"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [100, 149])
def test_an_infinity_enters_a_state(gpu, what, bad, at):
    """What the recurrence in 64 bits makes of a value that is not finite: infinities of either sign in
    the states and, behind (backward: before) that token, in the results that read them, NaN where it has
    NaN.  One state row or column is reached, the other entries are held to no bound here.
    (An infinite v in its own row: the recurrence sums q_d (k_d v), infinities of both signs, the chunk
    has (q . k) v, one infinity; both are the formula, so that row only has to be not finite.)"""
    lens = [150, 90]
    c = case(lens, 2, 64, 64, gpu, True, ld=torch.tensor([-0.02, -0.3]), seed=23)
    c[what][at, 1, 3] = bad
    do, q, k, v, ld, s0, ds = (c[s].cpu() for s in ("do", "q", "k", "v", "ld", "s0", "ds"))
    if what in "kv":
        o, out = run_fwd(c, gpu)
        want_o, want = recurrence(q, k, v, ld, lens, c["scale"], s0)
        rows, got_o = slice(at, 150), o
    else:
        _, gk, gv, out = run_bwd(c, gpu)
        _, want_k, want_v, want = reversed_recurrence(do, q, k, v, ld, lens, c["scale"], s0, ds)
        rows, got_o, want_o = slice(0, at + 1), gk if what == "do" else gv, want_k if what == "do" else want_v
    assert not torch.isfinite(want[0, 1]).all() and not torch.isfinite(want_o[rows, 1]).all()

    def wild(t):  # what is not finite, and which of the three
        return torch.where(torch.isfinite(t), torch.zeros_like(t), torch.where(torch.isnan(t), 2 + 0 * t.nan_to_num(0, 0, 0), t.sign()))
    assert torch.equal(wild(out.double().cpu()), wild(want))
    have, need = wild(got_o[rows, 1].double().cpu()), wild(want_o[rows, 1])
    if what == "v":
        assert torch.equal(have[0] != 0, need[0] != 0)
        have, need = have[1:], need[1:]
    assert torch.equal(have, need)


@pytest.mark.parametrize("lens", [[128], [64], [37], [100, 28]])
@pytest.mark.parametrize("d", [128, 64])
def test_a_state_keeps_24_bits(gpu, lens, d):
    """With keys (backward: queries) of a one and zeros, no two of d neighbours the same, a state's entry
    is the sum of one product or two (at d = 64), a value times a power of the decay.  It is held to the
    power's own error -- its exponent's roundings, two steps of fp32 for each of a chunk's three factors and
    their products, and for each chunk behind -- and the last bits of the product and its three parts."""
    c = case(lens, len(RATES), d, d, gpu, True, ld=torch.tensor(RATES), seed=24)
    c["s0"], c["ds"] = c["s0"] * 0, c["ds"] * 0
    t = torch.arange(c["n"], device=gpu) % d
    for s in "kq":
        c[s] = torch.nn.functional.one_hot(t, d)[:, None].expand(-1, len(RATES), -1).to(BF).contiguous()
    c["scale"] = 1.0
    _, out = run_fwd(c, gpu)
    gin = run_bwd(c, gpu)[3]
    do, q, k, v, ld, s0, ds = (c[s].cpu() for s in ("do", "q", "k", "v", "ld", "s0", "ds"))
    _, want = recurrence(q, k, v, ld, lens, 1.0, s0)
    *_, want_in = reversed_recurrence(do, q, k, v, ld, lens, 1.0, s0, ds)
    _, size = recurrence(q, k, v.abs(), ld, lens, 1.0, s0)
    *_, size_in = reversed_recurrence(do.abs(), q, k, v, ld, lens, 1.0, s0, ds)
    rate = torch.where(ld < -1e3, torch.zeros_like(ld), -ld).double()[:, None, None]
    err = F32 * (4 * rate * max(lens) + 16)
    check("state_out", out, want.to(gpu), (err * size + 2.0 ** -126 * 8).to(gpu))
    check("grad_state_in", gin, want_in.to(gpu), (err * size_in + 2.0 ** -126 * 8).to(gpu))
