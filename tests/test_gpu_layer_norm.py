"""The layer norm on the GPU against its formulas in 64 bits: widths of every kind
of lane group, rows apart, rows with a large mean, constant rows, infinities;
the backward against its formulas and against differences."""
from __future__ import annotations

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import F32, around_untouched, check, poisoned, rounded, spaced

pytestmark = pytest.mark.gpu
BF, FP, F4 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5
# fp32 additions that one value goes through in a row's sum: 16 in a lane, 6 among lanes, 16 waves
SUM = 40 * F32


def rows(n, d, dtype, dev, seed=0, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, d), generator=g) * (0.5 + torch.rand((n, 1), generator=g)) + mean
    return x.to(dtype).to(dev)


def weights(d, dev, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.2 * torch.randn(d, generator=g)).to(dev), (0.3 * torch.randn(d, generator=g)).to(dev)


def reference(x, w, b, eps=EPS):
    """y, mean, rstd and their bounds."""
    x, w = x.double(), w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    var = c.square().mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    emean = SUM * x.abs().mean(1, keepdim=True) + 2 * F32 * mean.abs()
    ec = emean + F32 * c.abs()
    evar = 2 * (c.abs() * ec).mean(1, keepdim=True) + ec.square().mean(1, keepdim=True) + SUM * var
    rel = evar / (var + eps) + 6 * F32  # of the deviation, at most
    u = c * rstd
    eu = rstd * ec * (1 + rel) + u.abs() * rel
    y = u * w + b
    ey = w.abs() * eu + 2 * F32 * (u * w).abs() + F32 * y.abs()
    return (y, ey), (mean[:, 0], emean[:, 0]), (rstd[:, 0], (rstd * rel)[:, 0])


WIDTHS = [8, 64, 72, 128, 200, 256, 264, 512, 520, 1024, 1032, 1368, 5120, 8192, 8200, 16384]


@pytest.mark.parametrize("dtype", [BF, FP, F4], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_forward(gpu, d, dtype):
    for n, bias, apart in ((1, True, False), (37, False, True), (130, True, True)):
        print(f"layer norm fwd n={n} d={d} {dtype} apart={apart}", flush=True)
        x, (w, b) = rows(n, d, dtype, gpu, seed=n), weights(d, gpu)
        b = b if bias else None
        xs = spaced(x, d + 24) if apart else x
        y, whole = poisoned((n, d), dtype, gpu, d + 16)
        saved = poisoned((n, 2), F4, gpu)
        eg.engram_layer_norm_fwd(xs, w, y, b=b, saved=saved, eps=EPS)
        torch.cuda.synchronize()
        (y64, ey), (m64, em), (r64, er) = reference(x, w, b)
        check("y", y, y64, ey + rounded(y64, dtype))
        check("mean", saved[:, 0], m64, em)
        check("rstd", saved[:, 1], r64, er)
        assert around_untouched(whole, d)
        y2 = poisoned((n, d), dtype, gpu)
        eg.engram_layer_norm_fwd(x, w, y2, b=b, eps=EPS)
        assert torch.equal(y2, y)


def backward(gy, x, w, saved, residual=None):
    """Gradients and bounds, from the saved moments as they are."""
    gy, x, w, mean, rstd = gy.double(), x.double(), w.double(), saved[:, :1].double(), saved[:, 1:].double()
    n = x.shape[0]
    u = (x - mean) * rstd
    eu = 2 * F32 * u.abs()
    g = gy * w
    m0, m1 = g.mean(1, keepdim=True), (g * u).mean(1, keepdim=True)
    a0, a1 = g.abs().mean(1, keepdim=True), (g * u).abs().mean(1, keepdim=True)
    gx = rstd * (g - m0 - u * m1)
    ex = rstd * (6 * F32 * (g.abs() + a0 + u.abs() * a1) + SUM * (a0 + u.abs() * a1) + 3 * F32 * u.abs() * a1)
    if residual is not None:
        gx = gx + residual.double()
        ex = ex + F32 * gx.abs()
    steps = (n / 512 + 80) * F32
    return (gx, ex), ((gy * u).sum(0), (steps + 3 * F32) * (gy * u).abs().sum(0)), (gy.sum(0), steps * gy.abs().sum(0))


@pytest.mark.parametrize("dtype", [BF, FP, F4], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_backward(gpu, d, dtype):
    for n, residual, apart in ((1, False, False), (37, True, True), (700, True, False)):
        print(f"layer norm bwd n={n} d={d} {dtype} apart={apart}", flush=True)
        x, gy, (w, _) = rows(n, d, dtype, gpu, seed=n), rows(n, d, dtype, gpu, seed=n + 1, mean=0), weights(d, gpu)
        r = rows(n, d, dtype, gpu, seed=n + 2) if residual else None
        _, (m, _), (s, _) = reference(x, w, None)
        saved = torch.stack((m, s), 1).float().contiguous()
        args = [spaced(t, d + 16) if apart and t is not None else t for t in (gy, x, r)]
        gx, whole = poisoned((n, d), dtype, gpu, d + 24)
        gw, gb = poisoned((d,), F4, gpu), poisoned((d,), F4, gpu)
        ws = poisoned((eg.engram_layer_norm_bwd_workspace_bytes(n, d),), torch.uint8, gpu)
        eg.engram_layer_norm_bwd(args[0], args[1], w, saved, gx, ws, grad_w=gw, grad_b=gb, grad_residual=args[2])
        torch.cuda.synchronize()
        (x64, ex), (w64, ew), (b64, eb) = backward(gy, x, w, saved, r)
        check("grad_x", gx, x64, ex + rounded(x64, dtype))
        check("grad_w", gw, w64, ew + 1e-37)
        check("grad_b", gb, b64, eb + 1e-37)
        assert around_untouched(whole, d)
        for kw in ({"grad_w": gw}, {"grad_b": gb}, {}):  # each weight gradient alone, and neither
            for t in kw.values():
                t.fill_(float("nan"))
            gx2 = poisoned((n, d), dtype, gpu)
            eg.engram_layer_norm_bwd(gy, x, w, saved, gx2, ws, grad_residual=r, **kw)
            assert torch.equal(gx2, gx)
        check("grad_w alone", gw, w64, ew + 1e-37)
        check("grad_b alone", gb, b64, eb + 1e-37)


def test_backward_against_differences(gpu):
    n, d, eps = 3, 72, 1e-3
    x, gy, (w, b) = rows(n, d, F4, gpu), rows(n, d, F4, gpu, seed=5), weights(d, gpu)
    saved, y, gx = torch.empty((n, 2), device=gpu), torch.empty_like(x), torch.empty_like(x)
    gw, gb = torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(eg.engram_layer_norm_bwd_workspace_bytes(n, d), dtype=torch.uint8, device=gpu)
    eg.engram_layer_norm_fwd(x, w, y, b=b, saved=saved, eps=EPS)
    eg.engram_layer_norm_bwd(gy, x, w, saved, gx, ws, grad_w=gw, grad_b=gb)
    g = torch.Generator().manual_seed(9)

    def loss(x_, w_, b_):
        return (reference(x_, w_, b_)[0][0] * gy.double()).sum()
    for name, grad in (("x", gx), ("w", gw), ("b", gb)):
        v = {"x": x.double(), "w": w.double(), "b": b.double()}
        for _ in range(6):
            d_ = torch.randn(grad.shape, generator=g, dtype=torch.float64).to(gpu)
            up, down = dict(v), dict(v)
            up[name], down[name] = v[name] + eps * d_, v[name] - eps * d_
            slope = (loss(up["x"], up["w"], up["b"]) - loss(down["x"], down["w"], down["b"])) / (2 * eps)
            # central differences: eps^2 times a third derivative of a few; fp32 gradients
            assert abs((grad.double() * d_).sum() - slope) <= 1e-4 * (grad.double() * d_).abs().sum(), name


@pytest.mark.parametrize("d", [64, 1024, 5120])
def test_rows_of_large_mean_and_constant_rows(gpu, d):
    x = rows(5, d, F4, gpu)
    x[1] += 10000.0
    x[2] = 3.7          # no deviation: y = b up to (x - mean) / sqrt(eps)
    x[3] = 0.0
    w, b = weights(d, gpu)
    y, saved = torch.empty_like(x), torch.empty((5, 2), device=gpu)
    eg.engram_layer_norm_fwd(x, w, y, b=b, saved=saved, eps=EPS)
    (y64, ey), (m64, em), _ = reference(x, w, b)
    check("y", y, y64, ey + rounded(y64, F4))
    check("mean", saved[:, 0], m64, em)
    assert torch.equal(y[3], b)


@pytest.mark.parametrize("d", [64, 5120])
def test_rows_that_are_not_finite_keep_to_themselves(gpu, d):
    x, gy = rows(9, d, BF, gpu), rows(9, d, BF, gpu, seed=3)
    w, b = weights(d, gpu)
    clean, saved = torch.empty_like(x), torch.empty((9, 2), device=gpu)
    eg.engram_layer_norm_fwd(x, w, clean, b=b, saved=saved)
    bad = x.clone()
    bad[2, 5], bad[7, 1] = float("inf"), float("nan")
    y = torch.empty_like(x)
    eg.engram_layer_norm_fwd(bad, w, y, b=b)
    keep = torch.tensor([i not in (2, 7) for i in range(9)], device=gpu)
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[[2, 7]]).all()
    ws = torch.empty(eg.engram_layer_norm_bwd_workspace_bytes(9, d), dtype=torch.uint8, device=gpu)
    gx, gx2 = torch.empty_like(x), torch.empty_like(x)
    eg.engram_layer_norm_bwd(gy, x, w, saved, gx, ws)
    gy[4, 0] = float("nan")
    eg.engram_layer_norm_bwd(gy, x, w, saved, gx2, ws)
    keep = torch.arange(9, device=gpu) != 4
    assert torch.equal(gx[keep], gx2[keep]) and torch.isnan(gx2[4]).all()


def test_captured_and_replayed_and_on_another_stream(gpu):
    n, d = 600, 1368
    x, gy, (w, b) = rows(n, d, BF, gpu), rows(n, d, BF, gpu, seed=4), weights(d, gpu)
    need = eg.engram_layer_norm_bwd_workspace_bytes(n, d)

    def buffers():
        return (torch.empty_like(x), torch.empty((n, 2), device=gpu), torch.empty_like(x), torch.empty_like(w),
                torch.empty_like(b), torch.empty(need, dtype=torch.uint8, device=gpu))

    def step(y, saved, gx, gw, gb, ws):
        eg.engram_layer_norm_fwd(x, w, y, b=b, saved=saved)
        eg.engram_layer_norm_bwd(gy, x, w, saved, gx, ws, grad_w=gw, grad_b=gb)
    want, kept, other = buffers(), buffers(), buffers()
    step(*want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*other)
    step(*want)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(i, j) for i, j in zip(want[:5], other[:5]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*kept)
    for _ in range(3):
        for t in kept[:5]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(want[:5], kept[:5]))
        step(*want)
