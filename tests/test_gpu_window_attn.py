"""The window attention on the GPU against its definition in 64 bits: ragged and
empty sequences, shared key heads, head sizes, windows from one token to all of
the past, sinks beside, inside and beyond the window, infinities that no row
sees, rows apart and rows behind the last sequence; the backward against its
formulas and against differences."""
from __future__ import annotations

import math

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import F32, HALF_STEP, around_untouched, check, poisoned, rounded, spaced

pytestmark = pytest.mark.gpu
BF, FP, F4 = torch.bfloat16, torch.float16, torch.float32


def visible(n, window, sinks):
    i = torch.arange(n)
    return (i[None, :] <= i[:, None]) & ((i[:, None] - i[None, :] < window) | (i[None, :] < sinks))


def case(lens, hq, hk, d, dtype, dev, window, sinks, tail=0, seed=0, apart=False, std=2.0):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens) + tail

    def r(*s):
        return torch.randn(s, generator=g)
    packed = r(n, (hq + 2 * hk) * d + 8)
    packed[:, :hq * d] *= std
    packed = packed.to(dtype).to(dev)
    q, k, v = (packed[:, x * d:(x + y) * d].unflatten(1, (y, d)) for x, y in ((0, hq), (hq, hk), (hq + hk, hk)))
    if not apart:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return {"q": q, "k": k, "v": v, "go": r(n, hq, d).to(dtype).to(dev), "lens": lens, "n": n, "b": len(lens), "hq": hq,
            "hk": hk, "d": d, "dtype": dtype, "window": window, "sinks": sinks, "scale": d ** -0.5,
            "cu": torch.tensor([0] + lens).cumsum(0).to(dev)}


def heads(c, rows, h):
    kh = h // (c["hq"] // c["hk"])
    return c["q"][rows, h].double(), c["k"][rows, kh].double(), c["v"][rows, kh].double(), kh


def weights(c, rows, h):
    """p, lse and the relative bound of a weight against exact ones."""
    q, k, v, kh = heads(c, rows, h)
    n = rows.stop - rows.start
    seen = visible(n, c["window"], c["sinks"]).to(q.device)
    z = (c["scale"] * (q @ k.t())).masked_fill(~seen, -math.inf)
    # a score is a sum of d exact products in fp32; scaled, and its maximum scaled, each a rounding
    za = c["scale"] * (q.abs() @ k.abs().t())
    ez = F32 * ((c["d"] + 4) * za.masked_fill(~seen, 0) + 4 * z.masked_fill(~seen, 0).abs().amax(1, keepdim=True))
    lse = torch.logsumexp(z, 1)
    p = torch.softmax(z, 1)
    rel = torch.expm1(2 * ez.amax(1, keepdim=True)) + F32 * (n + 8)
    return q, k, v, kh, p, lse, rel


def spans(c):
    at = 0
    for n in c["lens"]:
        if n:
            yield slice(at, at + n)
        at += n


def forward64(c):
    u = HALF_STEP[c["dtype"]]
    n, hq, d, dev = c["n"], c["hq"], c["d"], c["q"].device
    o, eo = (torch.zeros((n, hq, d), dtype=torch.float64, device=dev) for _ in range(2))
    lse, el = (torch.zeros((n, hq), dtype=torch.float64, device=dev) for _ in range(2))
    for rows in spans(c):
        for h in range(hq):
            _, _, v, _, p, ls, rel = weights(c, rows, h)
            o[rows, h] = p @ v
            # each weight rounded once, then fp32 sums; a weight rounded to fp16 may lose 2^-25 of the largest
            low = 2.0 ** -25 if c["dtype"] is FP else 0.0
            top = p.amax(1, keepdim=True)
            eo[rows, h] = (p @ v.abs()) * (u * (1 + rel) + rel + F32 * (rows.stop - rows.start + 8)) + low * top * v.abs().sum(0)
            lse[rows, h], el[rows, h] = ls, rel[:, 0] + 8 * F32 * (1 + ls.abs())
    return (o, eo + rounded(o, c["dtype"])), (lse, el)


def run_forward(c, dev, lse=True, stream=None):
    n, hq, d = c["n"], c["hq"], c["d"]
    o, whole = poisoned((n, hq, d), c["dtype"], dev, hq * d + 16)
    ls = poisoned((n, hq), F4, dev) if lse else None
    eg.engram_window_attn_fwd(c["q"], c["k"], c["v"], c["cu"], o, c["window"], sinks=c["sinks"], lse=ls, scale=c["scale"],
                              stream=stream)
    torch.cuda.synchronize()
    assert around_untouched(whole, hq * d)
    return o, ls


def backward64(c, o, lse, mean=False):
    """Gradients and bounds, given the forward's rounded o and lse; with `mean`, where delta is to be the weights' mean of
    the products with v, which keeps the digits that a rounded o has lost."""
    u = HALF_STEP[c["dtype"]]
    dev = c["q"].device
    gq, eq = (torch.zeros(c["q"].shape, dtype=torch.float64, device=dev) for _ in range(2))
    gk, ek, gv, ev = (torch.zeros(c["k"].shape, dtype=torch.float64, device=dev) for _ in range(4))
    for rows in spans(c):
        n = rows.stop - rows.start
        for h in range(c["hq"]):
            q, k, v, kh, p, ls, rel = weights(c, rows, h)
            g = c["go"][rows, h].double()
            # the kernel's weights come from the lse it is given, whose rounding (and bound) they carry
            off = rel + 2 * (lse[rows, h].double() - ls).abs()[:, None] + 4 * F32 * ls.abs()[:, None]
            dp, delta = g @ v.t(), (g * (p @ v)).sum(1, keepdim=True)
            # delta is the sum of g times the rounded o
            edelta = (g.abs() * (o[rows, h].double() - p @ v).abs()).sum(1, keepdim=True) + \
                F32 * (c["d"] + 8) * (g.abs() * o[rows, h].double().abs()).sum(1, keepdim=True)
            edp = F32 * (c["d"] + 4) * (g.abs() @ v.abs().t())
            if mean:  # a common factor of the weights cancels: their errors move the mean by what each is away from it
                edelta = 1.01 * (p * (off * (dp - delta).abs() + edp + F32 * (n + 8) * dp.abs())).sum(1, keepdim=True)
            ds = p * (dp - delta)
            eds = p * ((edp + edelta) * (1 + off) + off * (dp - delta).abs()) + 4 * F32 * ds.abs()
            tiny = 2.0 ** -25 if c["dtype"] is FP else 0.0  # what a weight or d rounded to fp16 may lose below its smallest steps
            eds = (eds + u * (ds.abs() + eds) + tiny * (p > 0)) * c["scale"]
            ep = p * (off + u * (1 + off)) + tiny * (p > 0)
            ds = ds * c["scale"]
            sums = F32 * (n * c["hq"] // c["hk"] + 70)
            gq[rows, h], eq[rows, h] = ds @ k, eds @ k.abs() + sums * (ds.abs() @ k.abs())
            gk[rows, kh] += ds.t() @ q
            ek[rows, kh] += eds.t() @ q.abs() + sums * (ds.abs().t() @ q.abs())
            gv[rows, kh] += p.t() @ g
            ev[rows, kh] += ep.t() @ g.abs() + sums * (p.t() @ g.abs())
    return [(x, e + rounded(x, c["dtype"])) for x, e in ((gq, eq), (gk, ek), (gv, ev))]


def run_backward(c, o, lse, dev):
    n, hq, hk, d, dt = c["n"], c["hq"], c["hk"], c["d"], c["dtype"]
    gq, whole_q = poisoned((n, hq, d), dt, dev, hq * d + 16)
    packed = poisoned((n, 2 * hk * d + 16), dt, dev)  # both gradients as columns of one row
    gk, gv = packed[:, 8:8 + hk * d].unflatten(1, (hk, d)), packed[:, 8 + hk * d:8 + 2 * hk * d].unflatten(1, (hk, d))
    ws = poisoned((eg.engram_window_attn_bwd_workspace_bytes(n, c["b"], hq, hk, d, c["window"], c["sinks"]),), torch.uint8, dev)
    eg.engram_window_attn_bwd(c["go"], c["q"], c["k"], c["v"], o, lse, c["cu"], gq, gk, gv, ws, c["window"], sinks=c["sinks"],
                              scale=c["scale"])
    torch.cuda.synchronize()
    assert around_untouched(whole_q, hq * d) and around_untouched(packed, 2 * hk * d)
    return gq, gk, gv


def check_all(c, dev):
    o, lse = run_forward(c, dev)
    m = sum(c["lens"])
    (o64, eo), (l64, el) = forward64(c)
    check("o", o[:m], o64[:m], eo[:m])
    check("lse", lse[:m], l64[:m], el[:m])
    assert torch.isnan(o[m:]).all() and torch.isnan(lse[m:]).all()  # rows behind the last sequence: left as they were
    o2, _ = run_forward(c, dev, lse=False)
    assert torch.equal(o2[:m], o[:m])
    got = run_backward(c, o, lse, dev)
    for name, g, (want, bound) in zip(("grad_q", "grad_k", "grad_v"), got, backward64(c, o, lse)):
        check(name, g[:m], want[:m], bound[:m])
        assert torch.isnan(g[m:]).all()


LENS = [[1], [63], [64], [65], [129], [300], [1, 0, 3, 64, 130, 0, 2], [0, 0, 5], [128, 128], [0], [1] * 20]
WINDOWS = [(1, 0), (5, 2), (64, 0), (100, 4), (37, 70), (1 << 40, 0), (200, 128)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
def test_forward_and_backward(gpu, lens, window, sinks):
    for hq, hk, d, dtype in ((6, 2, 128, BF), (2, 2, 64, FP)):
        print(f"window attn lens={lens} window={window} sinks={sinks} hq={hq} d={d} {dtype}", flush=True)
        check_all(case(lens, hq, hk, d, dtype, gpu, window, sinks, tail=3, apart=d == 128), gpu)


@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 1), (7, 7), (16, 2), (40, 8), (140, 1)])
@pytest.mark.parametrize("d", [8, 40, 64, 72, 80, 120, 128])
def test_heads(gpu, hq, hk, d):
    for dtype in (BF, FP):
        print(f"window attn heads {hq}/{hk} d={d} {dtype}", flush=True)
        check_all(case([90, 70], hq, hk, d, dtype, gpu, 50, 3, apart=True, seed=d), gpu)


@pytest.mark.parametrize("window,sinks", [(512, 4), (300, 128), (5000, 0)])
def test_long(gpu, window, sinks):
    """Several pieces of the sinks' sums, and of the rows behind a window."""
    check_all(case([2500, 700], 4, 2, 128, BF, gpu, window, sinks, seed=4), gpu)


@pytest.mark.parametrize("sinks", [1, 63, 64, 65, 127, 128])
def test_sinks_and_window_in_one_tile(gpu, sinks):
    check_all(case([400, 190], 4, 2, 72, BF, gpu, 30, sinks, seed=7), gpu)


@pytest.mark.parametrize("lens,window,sinks", [([2, 10, 3, 64], 64, 0), ([30, 128], 128, 0), ([200, 7], 50, 3)], ids=str)
def test_gradients_of_rows_that_see_few_keys(gpu, lens, window, sinks):
    """Up to two tiles of keys: the gradients are as exact as their own roundings, not as that of o."""
    for dtype in (BF, FP):
        c = case(lens, 2, 1, 128, dtype, gpu, window, sinks, seed=8)
        o, lse = run_forward(c, gpu)
        for name, g, (want, bound) in zip(("grad_q", "grad_k", "grad_v"), run_backward(c, o, lse, gpu),
                                          backward64(c, o, lse, mean=True)):
            print(f"window attn few keys {lens} {dtype} {name}", flush=True)
            check(name, g, want, bound)


def test_peaked_and_even_weights(gpu):
    for std in (0.0, 40.0):
        check_all(case([200], 2, 1, 64, BF, gpu, 64, 2, std=std, seed=5), gpu)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_what_a_row_does_not_see_does_not_reach_it(gpu, value, dtype):
    """Values that are not finite in one token's q, k, v or grad_o: every row that does not see it, and every token that
    it does not see, is as without it."""
    lens, at, window, sinks = [150, 200], 150 + 90, 40, 5
    c = case(lens, 4, 2, 72, dtype, gpu, window, sinks, seed=6)
    o, lse = run_forward(c, gpu)
    want = run_backward(c, o, lse, gpu)
    n = sum(lens)
    rows = torch.arange(n, device=gpu)
    sees = (rows >= at) & (rows < at + window)          # rows that see the token
    seen = (rows <= at) & (rows > at - window) | (rows >= 150) & (rows < 150 + sinks)  # tokens it sees
    (o64, eo), _ = forward64(c)
    # what the kernels sum row by row there, unrounded, is within the formulas' bounds
    bounds = [e for _, e in backward64(c, o, lse)]
    for name in ("k", "v", "q", "go"):
        b = {**c, name: c[name].clone()}
        b[name][at, :, 3] = value
        print(f"window attn {name} = {value} {dtype}", flush=True)
        if name in ("k", "v"):
            o2, _ = run_forward(b, gpu)
            check("o", o2[~sees], o64[~sees], eo[~sees])
            if name == "v":
                assert not torch.isfinite(o2[sees][:, :, 3]).any() and torch.isfinite(o2[sees][:, :, 4:]).all()
        got = run_backward(b, o, lse, gpu)
        # a key or value reaches dq of the rows that see it and its own dk and dv; a query or gradient its own dq, and
        # dk and dv of the tokens that it sees
        untouched = (~sees, rows != at, rows != at) if name in ("k", "v") else (rows != at, ~seen, ~seen)
        for x, w, e, ok in zip(got, want, bounds, untouched):
            check(name, x[ok], w[ok].double(), 2 * e[ok])


def test_bounds_outside_the_rows_are_clamped(gpu):
    c = case([50], 2, 1, 64, BF, gpu, 20, 2, seed=7)
    want, _ = run_forward(c, gpu)
    got, _ = run_forward({**c, "cu": torch.tensor([-7, 1 << 40], device=gpu)}, gpu)
    assert torch.equal(got, want)


def test_backward_against_differences(gpu):
    c = case([30, 9], 4, 2, 24, FP, gpu, 8, 2, seed=8)
    o, lse = run_forward(c, gpu)
    got = run_backward(c, o, lse, gpu)
    g = torch.Generator().manual_seed(1)
    base = {x: c[x].double() for x in "qkv"}

    def loss(v):
        (o64, _), _ = forward64({**c, **v})
        return (o64 * c["go"].double()).sum()
    for name, grad in zip("qkv", got):
        for _ in range(3):
            d = torch.randn(grad.shape, generator=g, dtype=torch.float64).to(gpu)
            eps = 1e-4
            slope = (loss({**base, name: base[name] + eps * d}) - loss({**base, name: base[name] - eps * d})) / (2 * eps)
            # the gradients' own roundings: a few half steps of fp16 (2^-11) of each term
            assert abs((grad.double() * d).sum() - slope) <= 2.0 ** -8 * (grad.double() * d).abs().sum(), name


def test_captured_and_replayed_and_two_streams(gpu):
    c = case([700, 333], 6, 2, 128, BF, gpu, 100, 4, seed=9)
    need = eg.engram_window_attn_bwd_workspace_bytes(c["n"], 2, 6, 2, 128, 100, 4)

    def buffers():
        return [torch.empty_like(c["q"]), torch.empty((c["n"], 6), device=gpu), torch.empty_like(c["q"]),
                torch.empty_like(c["k"]), torch.empty_like(c["v"]), torch.empty(need, dtype=torch.uint8, device=gpu)]

    def step(o, lse, gq, gk, gv, ws):
        eg.engram_window_attn_fwd(c["q"], c["k"], c["v"], c["cu"], o, 100, sinks=4, lse=lse, scale=c["scale"])
        eg.engram_window_attn_bwd(c["go"], c["q"], c["k"], c["v"], o, lse, c["cu"], gq, gk, gv, ws, 100, sinks=4,
                                  scale=c["scale"])
    want, other, again, kept = buffers(), buffers(), buffers(), buffers()
    step(*want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*other)
    step(*again)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(i, j) and torch.equal(i, k) for i, j, k in zip(want[:5], other[:5], again[:5]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*kept)
    for _ in range(3):
        for t in kept[:5]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(want[:5], kept[:5]))
        step(*again)
