"""The linear layer on the GPU against its definition in 64 bits: every path
(few rows, tiles of both sizes, a split contraction), every epilogue, ragged
sizes, rows apart; the backward against the formula and against differences."""
from __future__ import annotations

import math

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import F32, HALF_STEP, around_untouched, check, poisoned, rounded, spaced

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def inputs(n, k, m, dt, dev, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g, device=dev)
    return {"x": r(n, k).to(dt), "w": (r(m, k) * k ** -0.5).to(dt), "bias": r(m) * 0.5, "residual": r(n, m).to(dt),
            "grad_y": r(n, m).to(dt), "z": r(n, m).to(dt)}


def buffer(n, dev):
    return poisoned((n,), torch.uint8, dev) if n else None


# max |act'| is 1.13; the fp32 evaluation of act costs a few 2^-22 of |z| + 1 (an exponential, a division, and
# for gelu the approximation's 1.5e-7 of |z|)
ACT_SLOPE, ACT_ERR = 1.13, 2.0 ** -20


def fwd_bounds(d, act, bias, residual):
    x, w = d["x"].double(), d["w"].double()
    z = x @ w.t()
    zerr = F32 * (x.shape[1] + 2) * (x.abs() @ w.abs().t())
    if bias:
        z = z + d["bias"].double()
        zerr = zerr + F32 * z.abs()
    y, yerr = act64(z, act), zerr
    if act != "none":
        yerr = ACT_SLOPE * zerr + ACT_ERR * (1 + z.abs())
    if residual:
        y = y + d["residual"].double()
        yerr = yerr + F32 * y.abs()
    return z, zerr, y, yerr


FWD = [
    # n, k, m, dtype, act, bias, residual, z
    (1, 2560, 1024, BF, "none", False, False, False),
    (1, 8, 8, BF, "gelu", True, True, True),
    (2, 24, 40, FP, "silu", True, False, True),
    (7, 72, 1368, BF, "relu", False, True, False),
    (13, 5120, 136, FP, "silu", True, False, True),
    (16, 1000, 8200, BF, "none", True, True, False),      # 4 waves a workgroup
    (16, 640, 16392, BF, "gelu", True, False, False),     # 1024 workgroups and more
    (17, 128, 72, BF, "gelu", False, False, True),
    (32, 4168, 24, FP, "none", False, True, False),
    (33, 200, 520, BF, "silu", True, True, True),
    (64, 1032, 264, BF, "none", False, False, False),
    (64, 8, 16, FP, "relu", True, False, True),
    (65, 64, 128, BF, "none", False, False, False),       # tiles from here on
    (100, 4096, 256, BF, "silu", True, True, True),       # a split contraction
    (129, 4104, 136, FP, "gelu", True, False, False),
    (128, 8, 128, BF, "none", True, False, False),
    (300, 72, 1000, FP, "relu", False, True, True),
    (1025, 136, 392, BF, "gelu", True, True, False),
    (2049, 72, 6408, BF, "none", True, True, True),       # wide tiles
    (3333, 200, 4104, FP, "silu", False, False, False),
    (3333, 200, 4104, FP, "none", True, True, False),     # nothing but a residual (and bias) to add: wide tiles,
    (1500, 1032, 2568, BF, "none", False, True, False),   # ... two of 128 x 128 to a CU,
    (190, 264, 520, BF, "none", True, True, False),       # ... one,
    (100, 5000, 264, FP, "none", False, True, False),     # ... a split contraction
    (600, 5120, 264, BF, "none", False, False, False),    # parts for more than one round
]


@pytest.mark.parametrize("n,k,m,dt,act,bias,residual,z", FWD)
@pytest.mark.parametrize("apart", [False, True])
def test_forward(gpu, n, k, m, dt, act, bias, residual, z, apart):
    print(f"linear fwd n={n} k={k} m={m} {dt} {act} bias={bias} residual={residual} z={z} apart={apart}", flush=True)
    d = inputs(n, k, m, dt, gpu)
    z64, zerr, y64, yerr = fwd_bounds(d, act, bias, residual)
    if apart:
        x, res = spaced(d["x"], k + 24), spaced(d["residual"], m + 16)
        (y, whole), (zo, zwhole) = poisoned((n, m), dt, gpu, m + 40), poisoned((n, m), dt, gpu, m + 8)
    else:
        x, res = d["x"], d["residual"]
        y, zo = poisoned((n, m), dt, gpu), poisoned((n, m), dt, gpu)
    ws = buffer(eg.engram_linear_fwd_workspace_bytes(n, k, m), gpu)
    eg.engram_linear_fwd(x, d["w"], y, ws, bias=d["bias"] if bias else None, residual=res if residual else None,
                         z=zo if z else None, act=act)
    torch.cuda.synchronize()
    check("y", y, y64, rounded(y64, dt) * (1 + 2 * HALF_STEP[dt]) + yerr * (1 + HALF_STEP[dt]))
    if z:
        check("z", zo, z64, rounded(z64, dt) + 2 * zerr)
    if apart:
        assert around_untouched(whole, m)
        assert around_untouched(zwhole, m) or not z


BWD = [
    (1, 64, 8, BF, "none", True), (1, 2560, 1032, FP, "gelu", True), (13, 72, 264, BF, "silu", True),
    (64, 128, 128, BF, "relu", False), (65, 1000, 40, FP, "none", False), (200, 264, 520, BF, "gelu", True),
    (513, 8, 8, BF, "silu", True), (1000, 1032, 2056, FP, "relu", True), (2304, 4096, 264, BF, "none", True),
    (300, 4360, 3336, BF, "silu", False),
]


def bwd_bounds(d, act):
    x, w, g = d["x"].double(), d["w"].double(), d["grad_y"].double()
    n, k = x.shape
    m = w.shape[0]
    dt = d["x"].dtype
    dz, derr = g, torch.zeros_like(g)
    berr = torch.zeros_like(g)
    if act != "none":
        dz = g * slope64(d["z"].double(), act)
        berr = (ACT_ERR * (1 + d["z"].double().abs())) * g.abs()
        derr = rounded(dz, dt) + 1.01 * berr  # dz is rounded to the operands' type
    fx = (m + 2) * F32 * ((dz.abs() + derr) @ w.abs())
    fw = (n + 2) * F32 * ((dz.abs() + derr).t() @ x.abs())
    gx, gw, gb = dz @ w, dz.t() @ x, dz.sum(0)
    up = 1 + HALF_STEP[dt]
    return ((gx, rounded(gx, dt) + up * (fx + derr @ w.abs())), (gw, rounded(gw, dt) + up * (fw + derr.t() @ x.abs())),
            (gb, berr.sum(0) + (n + 2) * F32 * dz.abs().sum(0)))


def run_bwd(d, x, gy, act, gx, gw, gb, stream=None):
    n, k = d["x"].shape
    m = d["w"].shape[0]
    ws = buffer(eg.engram_linear_bwd_workspace_bytes(n, k, m), x.device)
    eg.engram_linear_bwd(gy, x, d["w"], gx, gw, ws, z=d["z"] if act != "none" else None, grad_bias=gb, act=act,
                         stream=stream)


@pytest.mark.parametrize("n,k,m,dt,act,bias", BWD)
@pytest.mark.parametrize("apart", [False, True])
def test_backward(gpu, n, k, m, dt, act, bias, apart):
    print(f"linear bwd n={n} k={k} m={m} {dt} {act} bias={bias} apart={apart}", flush=True)
    d = inputs(n, k, m, dt, gpu, seed=1)
    (gx64, bx), (gw64, bw), (gb64, bb) = bwd_bounds(d, act)
    x, gy = (spaced(d["x"], k + 8), spaced(d["grad_y"], m + 24)) if apart else (d["x"], d["grad_y"])
    gx, whole = poisoned((n, k), dt, gpu, k + 16)
    gw = poisoned((m, k), dt, gpu)
    gb = poisoned((m,), torch.float32, gpu) if bias else None
    run_bwd(d, x, gy, act, gx, gw, gb)
    torch.cuda.synchronize()
    check("grad_x", gx, gx64, bx)
    check("grad_w", gw, gw64, bw)
    if bias:
        check("grad_bias", gb, gb64, bb)
    assert around_untouched(whole, k)


def test_backward_of_parts(gpu):
    """Each output alone is what it is in the whole call, bit for bit."""
    d = inputs(70, 136, 264, BF, gpu, seed=2)
    whole = poisoned((70, 136), BF, gpu), poisoned((264, 136), BF, gpu), poisoned((264,), torch.float32, gpu)
    run_bwd(d, d["x"], d["grad_y"], "silu", *whole)
    for i in range(3):
        part = [poisoned(tuple(t.shape), t.dtype, gpu) if j == i else None for j, t in enumerate(whole)]
        run_bwd(d, d["x"], d["grad_y"], "silu", *part)
        torch.cuda.synchronize()
        assert torch.equal(part[i].view(torch.uint8), whole[i].view(torch.uint8))


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_backward_against_differences(gpu, act):
    """<gradient, direction> against (L(+h) - L(-h)) / 2h of the 64-bit forward, L = <y, grad_y>."""
    n, k, m = 37, 136, 72
    d = inputs(n, k, m, BF, gpu, seed=3)
    x, w, b, g = (d[s].double() for s in ("x", "w", "bias", "grad_y"))
    d["z"] = (x @ w.t() + b).to(BF)
    z = d["z"].double()  # the point at which the slopes are taken
    shift = z - (x @ w.t() + b)
    gx, gw, gb = poisoned((n, k), BF, gpu), poisoned((m, k), BF, gpu), poisoned((m,), torch.float32, gpu)
    run_bwd(d, d["x"], d["grad_y"], act, gx, gw, gb)
    bounds = bwd_bounds(d, act)
    gen = torch.Generator(device=gpu).manual_seed(4)
    for which, got, (_, bound) in (("x", gx, bounds[0]), ("w", gw, bounds[1]), ("bias", gb, bounds[2])):
        u = torch.randn(got.shape, generator=gen, device=gpu, dtype=torch.float64)
        h = 1e-5

        def loss(s):
            xx, ww, bb = x + (s * u if which == "x" else 0), w + (s * u if which == "w" else 0), b + (s * u if which == "bias" else 0)
            return (act64(xx @ ww.t() + bb + shift, act) * g).sum()
        want = ((loss(h) - loss(-h)) / (2 * h)).item()
        have = (got.double() * u).sum().item()
        # truncation: h^2 / 6 times a third derivative below |u|^3-sized sums; 1e-6 of the terms covers it and the cancellation
        assert abs(have - want) <= (bound * u.abs()).sum().item() + 1e-6 * (got.double() * u).abs().sum().item(), (which, have, want)


@pytest.mark.parametrize("n", [3, 40, 200])
def test_rows_are_independent(gpu, n):
    """A row of infinities or NaN leaves the others as they are, bit for bit."""
    d = inputs(n, 72, 136, BF, gpu, seed=5)

    def y(x):
        out = poisoned((n, 136), BF, gpu)
        eg.engram_linear_fwd(x, d["w"], out, buffer(eg.engram_linear_fwd_workspace_bytes(n, 72, 136), gpu), act="silu")
        return out
    clean = y(d["x"])
    x = d["x"].clone()
    x[1] = float("nan")
    x[n - 1] = float("inf")
    dirty = y(x)
    torch.cuda.synchronize()
    keep = [i for i in range(n) if i not in (1, n - 1)]
    assert torch.equal(clean[keep].view(torch.int16), dirty[keep].view(torch.int16))
    assert torch.isnan(dirty[1]).all()


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_activations_at_the_ends(gpu, act):
    """z = -inf, -1e30, -0, 0, 1e30, inf through the epilogue, and their slopes."""
    ends = torch.tensor([-math.inf, -1e30, -30.0, -0.0, 0.0, 30.0, 1e30, math.inf], device=gpu)
    x = torch.zeros((1, 8), dtype=BF, device=gpu)
    w = torch.zeros((8, 8), dtype=BF, device=gpu)
    y = poisoned((1, 8), BF, gpu)
    eg.engram_linear_fwd(x, w, y, bias=ends, act=act)
    want = torch.tensor([0, 0, 0, 0, 0, 30.0, 1e30, math.inf], device=gpu)
    torch.cuda.synchronize()
    assert torch.allclose(y[0].float(), want, rtol=2 ** -8, atol=1e-10), y
    gy = torch.ones((1, 8), dtype=BF, device=gpu)
    gb = poisoned((8,), torch.float32, gpu)
    ws = buffer(eg.engram_linear_bwd_workspace_bytes(1, 8, 8), gpu)
    z = ends.to(BF)[None]
    eg.engram_linear_bwd(gy, x, w, None, None, ws, z=z, grad_bias=gb, act=act)
    torch.cuda.synchronize()
    half = 0.0 if act == "relu" else 0.5
    assert torch.allclose(gb, torch.tensor([0, 0, 0, half, half, 1, 1, 1], device=gpu), atol=1e-6), gb


def test_relu_masks_infinite_gradients(gpu):
    """Where z is at most 0 nothing passes, also of an infinity or NaN in grad_y; a NaN in z passes on."""
    inf, nan = math.inf, math.nan
    z = torch.tensor([[-1.0, -0.0, 0.0, 2.0, -inf, inf, nan, 1.0]], device=gpu).to(BF)
    gy = torch.tensor([[inf, nan, -inf, 3.0, nan, 5.0, 7.0, -inf]], device=gpu).to(BF)
    w = torch.eye(8, device=gpu).to(BF)
    gb = poisoned((8,), torch.float32, gpu)
    ws = buffer(eg.engram_linear_bwd_workspace_bytes(1, 8, 8), gpu)
    eg.engram_linear_bwd(gy, torch.zeros((1, 8), dtype=BF, device=gpu), w, None, None, ws, z=z, grad_bias=gb, act="relu")
    torch.cuda.synchronize()
    assert gb.tolist() == [0.0, 0.0, 0.0, 3.0, 0.0, 5.0, 7.0, -inf], gb


def test_into_kv_and_through_the_gate(gpu):
    """The projections written straight into kv's columns feed the gate; the
    gate's grad_kv goes back through them: each step as if done alone."""
    n, k = 64, 264
    g = torch.Generator(device=gpu).manual_seed(6)

    def r(*s):
        return torch.randn(s, generator=g, device=gpu)
    mem, w = r(n, k).to(BF), (r(25600, k) * k ** -0.5).to(BF)
    x, weight = r(n, 4, 5120).to(BF), 1 + 0.1 * r(4, 5120)
    mask = torch.ones(n, dtype=torch.bool, device=gpu)
    mask[5] = False
    kv = poisoned((n, 25600), BF, gpu)
    for lo, hi in ((0, 20480), (20480, 25600)):  # keys, then the value
        m = hi - lo
        eg.engram_linear_fwd(mem, w[lo:hi], kv[:, lo:hi], buffer(eg.engram_linear_fwd_workspace_bytes(n, k, m), gpu))
    z64 = mem.double() @ w.double().t()
    check("kv", kv, z64, rounded(z64, BF) + 1.01 * F32 * (k + 2) * (mem.double().abs() @ w.double().abs().t()))
    out, saved = poisoned((n, 4, 5120), BF, gpu), poisoned((n, 4, 4), torch.float32, gpu)
    eg.engram_gate_fwd(x, kv, weight, mask, out, saved)
    assert torch.equal(out[5], x[5])
    gx, gkv, gw = poisoned((n, 4, 5120), BF, gpu), poisoned((n, 25600), BF, gpu), poisoned((4, 5120), torch.float32, gpu)
    eg.engram_gate_bwd(x, kv, weight, saved, r(n, 4, 5120).to(BF), gx, gkv, gw,
                       buffer(eg.engram_gate_bwd_workspace_bytes(n), gpu))
    d = {"x": mem, "w": w, "grad_y": gkv, "z": gkv}
    gmem, gwk = poisoned((n, k), BF, gpu), poisoned((25600, k), BF, gpu)
    run_bwd(d, mem, gkv, "none", gmem, gwk, None)
    torch.cuda.synchronize()
    bounds = bwd_bounds(d, "none")
    check("grad_mem", gmem, *bounds[0])
    check("grad_w", gwk, *bounds[1])


def test_graph_and_streams(gpu):
    """Forward and backward captured once and replayed, eager work in between,
    and the same calls on two other streams at once: bit for bit the eager results."""
    n, k, m = 100, 1032, 264
    d = inputs(n, k, m, BF, gpu, seed=7)

    def make():
        return {"y": poisoned((n, m), BF, gpu), "z": poisoned((n, m), BF, gpu), "gx": poisoned((n, k), BF, gpu),
                "gw": poisoned((m, k), BF, gpu), "gb": poisoned((m,), torch.float32, gpu),
                "wf": buffer(eg.engram_linear_fwd_workspace_bytes(n, k, m), gpu),
                "wb": buffer(eg.engram_linear_bwd_workspace_bytes(n, k, m), gpu)}

    def go(o, stream=None):
        eg.engram_linear_fwd(d["x"], d["w"], o["y"], o["wf"], bias=d["bias"], z=o["z"], act="gelu", stream=stream)
        eg.engram_linear_bwd(d["grad_y"], d["x"], d["w"], o["gx"], o["gw"], o["wb"], z=o["z"], grad_bias=o["gb"],
                             act="gelu", stream=stream)

    def same(a, b):
        return all(torch.equal(a[s].view(torch.uint8), b[s].view(torch.uint8)) for s in ("y", "z", "gx", "gw", "gb"))
    want, got = make(), make()
    go(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(got)
    for _ in range(3):
        for s in got.values():
            if s is not None:
                s.view(torch.uint8).fill_(0xFF)
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
