"""The norms of queries and keys with the rotation, on the GPU, against the
definition in 64 bits: head sizes and layouts, pairings, element types, far
and negative positions, rows apart; the backward against the formula and
against differences."""
from __future__ import annotations

import math

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import F32, HALF_STEP, around_untouched, check, poisoned, rounded

pytestmark = pytest.mark.gpu
BF, FP, F4 = torch.bfloat16, torch.float16, torch.float32
THETA, EPS = 10000.0, 1e-6
# the rotation's error: the 32-bit fraction of a turn rounded to fp32 (2^-25 of half a turn) times 2 pi, and the
# sine's and cosine's own: the hardware's for 16-bit outputs (a few 2^-20), the library's for fp32 (a few 2^-24)
ANGLE = {BF: 2.0 ** -17, FP: 2.0 ** -17, F4: 2.0 ** -21}


def factors(positions, r):
    """cos, sin [N, 1, R/2] in 64 bits; positions below 2^53 / R keep them exact enough only for small angles, so
    the angle is reduced in whole turns with integers first: the table's 64-bit fractions."""
    table = eg.engram_rope_freqs(THETA, r).tolist()
    turns = torch.tensor([[((p * f) & (2 ** 64 - 1)) / 2.0 ** 64 for f in table] for p in positions.tolist()],
                         dtype=torch.float64)
    a = 2 * math.pi * turns[:, None]
    return torch.cos(a).to(positions.device), torch.sin(a).to(positions.device)


def pair_index(r, interleaved, dev):
    i = torch.arange(r // 2, device=dev)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)


def turn(y, cos, sin, r, interleaved):
    if r == 0:
        return y
    p, q = pair_index(r, interleaved, y.device)
    out = y.clone()
    out[..., p] = y[..., p] * cos - y[..., q] * sin
    out[..., q] = y[..., p] * sin + y[..., q] * cos
    return out


def partner_abs(y, r, interleaved):
    """|y| plus its pair partner's."""
    out = y.abs().clone()
    if r:
        p, q = pair_index(r, interleaved, y.device)
        both = y[..., p].abs() + y[..., q].abs()
        out[..., p], out[..., q] = both, both
    return out


def forward64(x, w, cos, sin, r, interleaved, eps=EPS):
    rstd = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return turn(x * rstd * w, cos, sin, r, interleaved)


def case(n, hq, hk, d, r, dt, dev, apart=False, seed=0, far=1 << 20):
    g = torch.Generator(device=dev).manual_seed(seed)
    packed = torch.randn((n, (hq + 2 * hk) * d + (16 if apart else 0)), generator=g, device=dev).to(dt)
    c = {"q": packed[:, :hq * d].unflatten(1, (hq, d)), "k": packed[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))}
    if not apart:
        c = {s: t.contiguous() for s, t in c.items()}
    c["wq"], c["wk"] = (1 + 0.3 * torch.randn((d,), generator=g, device=dev) for _ in range(2))
    c["positions"] = torch.randint(-far, far, (n,), generator=g, device=dev)
    c["freqs"] = eg.engram_rope_freqs(THETA, r).to(dev) if r else None
    c["gq"], c["gk"] = (torch.randn((n, h, d), generator=g, device=dev).to(dt) for h in (hq, hk))
    return c


CASES = [
    # n, hq, hk, d, r, interleaved, dtype
    (1, 40, 8, 128, 128, False, BF), (16, 40, 8, 128, 128, False, BF), (3, 1, 1, 8, 0, False, F4),
    (5, 3, 2, 16, 16, False, BF), (7, 5, 1, 40, 32, True, FP), (33, 12, 3, 80, 48, False, F4),
    (130, 4, 4, 64, 64, True, BF), (9, 9, 7, 96, 96, False, FP), (2, 2, 1, 256, 128, False, BF),
    (3, 2, 2, 512, 512, True, F4), (4, 3, 1, 504, 496, False, FP), (1100, 2, 1, 128, 64, True, BF),
    (2500, 16, 2, 72, 64, False, BF), (6, 33, 17, 24, 16, False, BF),
]


@pytest.mark.parametrize("n,hq,hk,d,r,inter,dt", CASES)
@pytest.mark.parametrize("apart", [False, True])
def test_forward(gpu, n, hq, hk, d, r, inter, dt, apart):
    print(f"qk fwd n={n} hq={hq} hk={hk} d={d} r={r} inter={inter} {dt} apart={apart}", flush=True)
    c = case(n, hq, hk, d, r, dt, gpu, apart)
    cos, sin = factors(c["positions"], r) if r else (None, None)
    if apart:  # both outputs are columns of one packed row
        _, whole = poisoned((n, (hq + hk) * d), dt, gpu, (hq + hk) * d + 24)
        qo = whole[:, 8:8 + hq * d].unflatten(1, (hq, d))
        ko = whole[:, 8 + hq * d:8 + (hq + hk) * d].unflatten(1, (hk, d))
    else:
        qo, ko = poisoned((n, hq, d), dt, gpu), poisoned((n, hk, d), dt, gpu)
    eg.engram_qk_norm_rope_fwd(c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["freqs"], qo, ko, eps=EPS,
                               interleaved=inter)
    torch.cuda.synchronize()
    for name, x, w, got in (("q_out", c["q"], c["wq"], qo), ("k_out", c["k"], c["wk"], ko)):
        x, w = x.double(), w.double()
        want = forward64(x, w, cos, sin, r, inter)
        y = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
        # mean of d squares, root, reciprocal, two products, the rotation
        bound = rounded(want, dt) + (F32 * (d + 8) + ANGLE[dt]) * partner_abs(y, r, inter) * (1 + HALF_STEP[dt])
        check(name, got, want, bound)
    if apart:
        assert around_untouched(whole, (hq + hk) * d)


def backward64(g, x, w, cos, sin, r, interleaved, eps=EPS):
    g = turn(g, cos, None if sin is None else -sin, r, interleaved)
    rstd = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    u, gw = x * rstd, g * w
    return rstd * (gw - u * (u * gw).mean(-1, keepdim=True)), (g * u).sum((0, 1)), g, u, rstd


def bwd_bounds(g, x, w, cos, sin, r, inter, dt):
    n, h, d = x.shape
    dx, dw, gr, u, rstd = backward64(g.double(), x.double(), w.double(), cos, sin, r, inter)
    gerr = (ANGLE[dt] + 8 * F32) * partner_abs(g.double(), r, inter)
    gwa = (gr.abs() + gerr) * w.double().abs()
    small = F32 * (2 * d + 16)
    part = u.abs() * (u.abs() * gwa).mean(-1, keepdim=True)
    perr = u.abs() * (u.abs() * gerr * w.double().abs()).mean(-1, keepdim=True)
    dxerr = rstd * (gerr * w.double().abs() + perr + small * (gwa + part))
    terms = (gr.abs() + gerr) * u.abs()
    dwerr = (gerr * u.abs()).sum((0, 1)) + F32 * (d + 16 + n * h / 4 + 40) * terms.sum((0, 1))
    return (dx, rounded(dx, dt) + (1 + HALF_STEP[dt]) * dxerr), (dw, dwerr)


def run_bwd(c, inter, dt, gpu, packed=False):
    n, hq, d = c["q"].shape
    hk = c["k"].shape[1]
    if packed:
        _, whole = poisoned((n, (hq + hk) * d), dt, gpu, (hq + hk) * d + 8)
        gq, gk = whole[:, 8:8 + hq * d].unflatten(1, (hq, d)), whole[:, 8 + hq * d:].unflatten(1, (hk, d))
    else:
        gq, gk = poisoned((n, hq, d), dt, gpu), poisoned((n, hk, d), dt, gpu)
    gwq, gwk = poisoned((d,), F4, gpu), poisoned((d,), F4, gpu)
    ws = poisoned((eg.engram_qk_norm_rope_bwd_workspace_bytes(n, hq, hk, d),), torch.uint8, gpu)
    eg.engram_qk_norm_rope_bwd(c["gq"], c["gk"], c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["freqs"], gq, gk,
                               gwq, gwk, ws, eps=EPS, interleaved=inter)
    torch.cuda.synchronize()
    return gq, gk, gwq, gwk


@pytest.mark.parametrize("n,hq,hk,d,r,inter,dt", CASES)
@pytest.mark.parametrize("apart", [False, True])
def test_backward(gpu, n, hq, hk, d, r, inter, dt, apart):
    print(f"qk bwd n={n} hq={hq} hk={hk} d={d} r={r} inter={inter} {dt} apart={apart}", flush=True)
    c = case(n, hq, hk, d, r, dt, gpu, apart, seed=1)
    cos, sin = factors(c["positions"], r) if r else (None, None)
    gq, gk, gwq, gwk = run_bwd(c, inter, dt, gpu, packed=apart)
    for s, gx, gw in (("q", gq, gwq), ("k", gk, gwk)):
        bx, bw = bwd_bounds(c["g" + s], c[s], c["w" + s], cos, sin, r, inter, dt)
        check("grad_" + s, gx, *bx)
        check("grad_w" + s, gw, *bw)


@pytest.mark.parametrize("inter", [False, True])
def test_backward_against_differences(gpu, inter):
    n, hq, hk, d, r = 5, 3, 2, 40, 32
    c = case(n, hq, hk, d, r, F4, gpu, seed=2)
    cos, sin = factors(c["positions"], r)
    gq, gk, gwq, gwk = run_bwd(c, inter, F4, gpu)
    gen = torch.Generator(device=gpu).manual_seed(3)
    for s, gx, gw in (("q", gq, gwq), ("k", gk, gwk)):
        x, w, g = c[s].double(), c["w" + s].double(), c["g" + s].double()
        for at, got in (("x", gx), ("w", gw)):
            u = torch.randn(got.shape, generator=gen, device=gpu, dtype=torch.float64)
            h = 1e-5
            lo, hi = ((forward64(x + (t * u if at == "x" else 0), w + (t * u if at == "w" else 0), cos, sin, r, inter) * g).sum()
                      for t in (-h, h))
            want, have = ((hi - lo) / (2 * h)).item(), (got.double() * u).sum().item()
            assert abs(have - want) <= 2e-5 * (got.double() * u).abs().sum().item(), (s, at, have, want)


def test_far_positions(gpu):
    """Positions where a 32-bit, and a 64-bit floating, angle would have lost every bit of its fraction."""
    n, d = 6, 64
    c = case(n, 2, 1, d, d, F4, gpu, seed=4)
    c["positions"] = torch.tensor([0, 1, -1, 2 ** 31 + 7, 2 ** 53 + 1, 2 ** 62 + 12345], device=gpu)
    cos, sin = factors(c["positions"], d)
    qo, ko = poisoned((n, 2, d), F4, gpu), poisoned((n, 1, d), F4, gpu)
    eg.engram_qk_norm_rope_fwd(c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["freqs"], qo, ko)
    torch.cuda.synchronize()
    y = forward64(c["q"].double(), c["wq"].double(), cos, sin, 0, False)
    want = turn(y, cos, sin, d, False)
    check("q_out", qo, want, (F32 * (d + 8) + ANGLE[F4]) * partner_abs(y, d, False))
    rest = c["q"].double() * (c["q"].double().square().mean(-1, keepdim=True) + EPS).rsqrt() * c["wq"].double()
    check("position 0", qo[:1], rest[:1], F32 * (d + 8) * partner_abs(rest[:1], d, False) + 1e-30)


def test_table_matches_64_bits():
    for theta, r in ((10000.0, 128), (500000.0, 64), (2.0, 16), (1.0, 32)):
        t = eg.engram_rope_freqs(theta, r).tolist()
        assert len(t) == r // 2
        for i, f in enumerate(t):
            want = theta ** (-2.0 * i / r) / (2 * math.pi)
            # half a step of the table, and a few steps of the 64-bit power it is compared with
            assert abs((f & (2 ** 64 - 1)) / 2.0 ** 64 - want) <= 2.0 ** -65 + 2.0 ** -50 * want


@pytest.mark.parametrize("dt", [BF, F4])
def test_zero_tiny_and_non_finite_heads(gpu, dt):
    """A head of zeros gives zeros (and a finite gradient); heads of infinities or NaN leave the others alone."""
    c = case(4, 3, 1, 64, 64, dt, gpu, seed=5)
    clean_q, clean_k = poisoned((4, 3, 64), dt, gpu), poisoned((4, 1, 64), dt, gpu)

    def go(qo, ko):
        eg.engram_qk_norm_rope_fwd(c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["freqs"], qo, ko)
        torch.cuda.synchronize()
    go(clean_q, clean_k)
    c["q"][0, 0] = 0
    c["q"][1, 1] = float("inf")
    c["q"][2, 2, 5] = float("nan")
    c["q"][3, 0] = 1e-30
    qo, ko = poisoned((4, 3, 64), dt, gpu), poisoned((4, 1, 64), dt, gpu)
    go(qo, ko)
    assert (qo[0, 0] == 0).all()
    assert torch.isnan(qo[2, 2]).all() and torch.isnan(qo[1, 1]).all()
    assert torch.isfinite(qo[3, 0]).all()
    keep = torch.ones((4, 3), dtype=torch.bool, device=gpu)
    keep[0, 0] = keep[1, 1] = keep[2, 2] = keep[3, 0] = False
    assert torch.equal(qo[keep].view(torch.uint8), clean_q[keep].view(torch.uint8))
    assert torch.equal(ko.view(torch.uint8), clean_k.view(torch.uint8))
    c["q"][1, 1] = 1
    c["q"][2, 2] = 1
    for t in run_bwd(c, False, dt, gpu):
        assert torch.isfinite(t).all()


def test_graph_and_streams(gpu):
    c = case(50, 6, 2, 128, 64, BF, gpu, seed=6)

    def make():
        return {"qo": poisoned((50, 6, 128), BF, gpu), "ko": poisoned((50, 2, 128), BF, gpu),
                "gq": poisoned((50, 6, 128), BF, gpu), "gk": poisoned((50, 2, 128), BF, gpu),
                "gwq": poisoned((128,), F4, gpu), "gwk": poisoned((128,), F4, gpu),
                "ws": poisoned((eg.engram_qk_norm_rope_bwd_workspace_bytes(50, 6, 2, 128),), torch.uint8, gpu)}

    def go(o, stream=None):
        args = (c["q"], c["k"], c["wq"], c["wk"], c["positions"], c["freqs"])
        eg.engram_qk_norm_rope_fwd(*args, o["qo"], o["ko"], stream=stream)
        eg.engram_qk_norm_rope_bwd(c["gq"], c["gk"], *args, o["gq"], o["gk"], o["gwq"], o["gwk"], o["ws"], stream=stream)

    def same(a, b):
        return all(torch.equal(a[s].view(torch.uint8), b[s].view(torch.uint8)) for s in a if s != "ws")
    want, got = make(), make()
    go(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(got)
    for _ in range(3):
        for t in got.values():
            t.view(torch.uint8).fill_(0xFF)
        torch.randn(1000, device=gpu).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, got)
    streams, sets = [torch.cuda.Stream() for _ in range(2)], [make(), make()]
    torch.cuda.synchronize()
    for st, o in zip(streams, sets):
        go(o, stream=st)
    torch.cuda.synchronize()
    assert same(want, sets[0]) and same(want, sets[1])
