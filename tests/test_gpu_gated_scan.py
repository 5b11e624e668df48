"""The gated recurrence on the GPU against its definition in 64 bits, token after
token: ragged and empty sequences, carried states, widths, gates from shut to
open, many chunks, infinities, rows behind the last sequence; the backward
against the reversed recurrence and against differences; the step, with a
slot more than once."""
from __future__ import annotations

import math

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import F32, around_untouched, check, poisoned, rounded, spaced

pytestmark = pytest.mark.gpu
BF, FP, F4 = torch.bfloat16, torch.float16, torch.float32


def gates(g):
    """f, 1 - f and the bound of the smaller one: exp2's argument in fp32 is off by 2^-24 of itself and by
    log2(e)'s own rounding, exp2 and the reciprocal by a step each, then a product; and where it is below 2^-126
    (gates beyond 87) exp2 gives 0, off by less than 2^-126."""
    g = g.double()
    f, n = torch.sigmoid(g), torch.sigmoid(-g)
    return f, n, F32 * (2 * g.abs() + 8) * torch.minimum(f, n) + 2.0 ** -126


def spans(lens):
    at = 0
    for b, n in enumerate(lens):
        yield b, at, at + n
        at += n


def recurrence(gate, u, lens, s0):
    """h and last states with bounds: e is the error carried along, beside a, the recurrence over absolute values."""
    f, n, off = gates(gate)
    u = u.double()
    h, eh = torch.zeros_like(u), torch.zeros_like(u)
    out = torch.zeros((len(lens), u.shape[1]), dtype=torch.float64, device=u.device)
    eout = torch.zeros_like(out)
    for b, lo, hi in spans(lens):
        s = torch.zeros_like(out[0]) if s0 is None else s0[b].double()
        a, e = s.abs(), torch.zeros_like(s)
        for t in range(lo, hi):
            # s x of the smaller factor, and at most eight roundings of what there is, the chunks' products among them
            e = f[t] * e + off[t] * (a + u[t].abs()) + 8 * F32 * (f[t] * a + n[t] * u[t].abs())
            a = f[t] * a + n[t] * u[t].abs()
            s = f[t] * s + n[t] * u[t]
            h[t], eh[t] = s, e
        out[b], eout[b] = s, e
    return (h, eh), (out, eout)


def reversed_recurrence(gh, gate, u, h, lens, s0, ds):
    f, n, off = gates(gate)
    gh, u, h = gh.double(), u.double(), h.double()
    dg, eg_, du, eu = (torch.zeros_like(u) for _ in range(4))
    out = torch.zeros((len(lens), u.shape[1]), dtype=torch.float64, device=u.device)
    eout = torch.zeros_like(out)
    for b, lo, hi in spans(lens):
        c = torch.zeros_like(out[0]) if ds is None else ds[b].double()
        a, e = c.abs(), torch.zeros_like(c)
        for t in reversed(range(lo, hi)):
            dh, adh, edh = gh[t] + c, gh[t].abs() + a, e + F32 * (gh[t].abs() + a)
            before = h[t - 1] if t > lo else (torch.zeros_like(c) if s0 is None else s0[b].double())
            k = f[t] * n[t] * (before - u[t])
            dg[t], du[t] = dh * k, dh * n[t]
            eg_[t] = edh * k.abs() + adh * (before - u[t]).abs() * (2 * off[t] + 8 * F32 * f[t] * n[t])
            eu[t] = edh * n[t] + adh * (off[t] + 3 * F32 * n[t])
            c, a = f[t] * dh, f[t] * adh
            e = f[t] * edh + off[t] * adh + 8 * F32 * f[t] * adh
        out[b], eout[b] = c, e
    return (dg, eg_), (du, eu), (out, eout)


def case(lens, d, dtype, dev, states, tail=0, seed=0, apart=False, bias=2.0):
    g = torch.Generator().manual_seed(seed)
    n, b = sum(lens) + tail, len(lens)

    def r(*s):
        return torch.randn(s, generator=g)
    packed = r(n, 2 * d + 8)
    packed[:, :d] += bias * torch.linspace(-1, 2, d)
    packed = packed.to(dtype).to(dev)
    gate, u = packed[:, :d], packed[:, d:2 * d]
    if not apart:
        gate, u = gate.contiguous(), u.contiguous()
    return {"gate": gate, "u": u, "gh": r(n, d).to(dtype).to(dev), "lens": lens, "n": n, "b": b, "d": d, "dtype": dtype,
            "cu": torch.tensor([0] + lens).cumsum(0).to(dev), "s0": r(b, d).to(dev) if states else None,
            "ds": r(b, d).to(dev) if states else None}


def forward(c, dev, stream=None):
    n, b, d = c["n"], c["b"], c["d"]
    h, whole = poisoned((n, d), c["dtype"], dev, d + 16)
    out = poisoned((b, d), F4, dev)
    ws = poisoned((eg.engram_gated_scan_fwd_workspace_bytes(n, b, d),), torch.uint8, dev)
    eg.engram_gated_scan_fwd(c["gate"], c["u"], c["cu"], h, ws, state_in=c["s0"], state_out=out, stream=stream)
    torch.cuda.synchronize()
    assert around_untouched(whole, d)
    return h, out


def backward(c, h, dev):
    n, b, d, dtype = c["n"], c["b"], c["d"], c["dtype"]
    gg, whole = poisoned((n, d), dtype, dev, d + 16)
    gu, gin = poisoned((n, d), dtype, dev), poisoned((b, d), F4, dev)
    ws = poisoned((eg.engram_gated_scan_bwd_workspace_bytes(n, b, d),), torch.uint8, dev)
    eg.engram_gated_scan_bwd(c["gh"], c["gate"], c["u"], h, c["cu"], gg, gu, ws, state_in=c["s0"], grad_state_out=c["ds"],
                             grad_state_in=gin)
    torch.cuda.synchronize()
    assert around_untouched(whole, d)
    return gg, gu, gin


def check_forward(c, dev):
    h, out = forward(c, dev)
    m = sum(c["lens"])
    cpu = {k: None if c[k] is None else c[k].cpu() for k in ("gate", "u", "s0")}
    (h64, eh), (s64, es) = recurrence(cpu["gate"][:m], cpu["u"][:m], c["lens"], cpu["s0"])
    check("h", h[:m], h64.to(dev), (eh + rounded(h64, c["dtype"])).to(dev))
    check("state_out", out, s64.to(dev), (es + F32 * s64.abs() + 1e-37).to(dev))
    assert torch.isnan(h[m:]).all()  # rows behind the last sequence: left as they were
    return h


def check_backward(c, h, dev):
    gg, gu, gin = backward(c, h, dev)
    m = sum(c["lens"])
    cpu = {k: None if c[k] is None else c[k].cpu() for k in ("gh", "gate", "u", "s0", "ds")}
    (g64, eg_), (u64, eu), (s64, es) = reversed_recurrence(cpu["gh"][:m], cpu["gate"][:m], cpu["u"][:m], h[:m].cpu(), c["lens"],
                                                           cpu["s0"], cpu["ds"])
    check("grad_gate", gg[:m], g64.to(dev), (eg_ + rounded(g64, c["dtype"])).to(dev))
    check("grad_u", gu[:m], u64.to(dev), (eu + rounded(u64, c["dtype"])).to(dev))
    check("grad_state_in", gin, s64.to(dev), (es + F32 * s64.abs() + 1e-37).to(dev))
    assert torch.isnan(gg[m:]).all() and torch.isnan(gu[m:]).all()


# chunks have 32 tokens (fp32) or 64, groups eight chunks: 256 or 512 tokens
LENS = [[1], [3], [8], [32], [33], [64], [65], [16, 16, 1], [255], [256], [257], [512], [513], [1, 0, 3, 64, 129, 0, 2], [0, 0, 5], [0], [700],
        [1] * 70, [300, 0, 1, 511, 7]]


@pytest.mark.parametrize("dtype", [BF, FP, F4], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_forward_and_backward(gpu, lens, dtype):
    for d, states in ((72, True), (8, False), (1032, True)):
        print(f"gated scan lens={lens} d={d} {dtype} states={states}", flush=True)
        c = case(lens, d, dtype, gpu, states, tail=5, apart=states, seed=d)
        h = check_forward(c, gpu)
        check_backward(c, h, gpu)


@pytest.mark.parametrize("dtype", [BF, F4], ids=["bf16", "fp32"])
def test_many_chunks(gpu, dtype):
    """Far more workgroups than the chip holds at once, and several spans of eight groups (2048 or 4096 tokens) in one
    sequence, one that begins inside a span and one that ends with one."""
    c = case([9000, 3288, 41], 2056, dtype, gpu, True, seed=2)
    h = check_forward(c, gpu)
    check_backward(c, h, gpu)


@pytest.mark.parametrize("bias", [-100.0, -30.0, 0.0, 12.0, 30.0, 120.0])
def test_gates_from_shut_to_open(gpu, bias):
    c = case([200, 60], 64, F4, gpu, True, seed=3)
    c["gate"] = (c["gate"] * 0.1 + bias).contiguous()
    h = check_forward(c, gpu)
    check_backward(c, h, gpu)


def test_extreme_gates(gpu):
    """Infinite gates: nothing kept, or everything."""
    c = case([100], 16, F4, gpu, True, seed=4)
    c["gate"][:, :8], c["gate"][:, 8:] = math.inf, -math.inf
    h, out = forward(c, gpu)
    assert torch.equal(h[:, :8], c["s0"][:, :8].expand(100, 8)) and torch.equal(h[:, 8:], c["u"][:, 8:])
    assert torch.equal(out[0], h[-1])


def test_an_infinite_input_stays_with_its_sequence_and_channel(gpu):
    lens = [40, 90, 50]
    c = case(lens, 16, BF, gpu, True, seed=5)
    clean, _ = forward(c, gpu)
    c["u"][60, 3], c["u"][70, 5], c["gate"][100, 7] = math.inf, -math.inf, math.nan
    h, out = forward(c, gpu)
    touched = torch.zeros_like(h, dtype=torch.bool)
    touched[60:130, 3] = touched[70:130, 5] = touched[100:130, 7] = True
    assert torch.equal(h[~touched], clean[~touched])
    assert (h[60:130, 3] == math.inf).all() and (h[70:130, 5] == -math.inf).all() and torch.isnan(h[100:130, 7]).all()
    assert out[1, 3] == math.inf and out[1, 5] == -math.inf and torch.isnan(out[1, 7]) and torch.isfinite(out[2]).all()
    c = case(lens, 16, BF, gpu, True, seed=5)
    h, _ = forward(c, gpu)
    want = backward(c, h, gpu)
    c["gh"][100, 2], c["gh"][60, 4] = math.inf, math.nan
    got = backward(c, h, gpu)
    touched.zero_()
    touched[40:101, 2] = touched[40:61, 4] = True
    for g, w in zip(got[:2], want[:2]):
        assert torch.equal(g[~touched], w[~touched]) and not torch.isfinite(g[touched]).any()
    assert got[2][1, 2] == math.inf and torch.isnan(got[2][1, 4]) and torch.equal(got[2][[0, 2]], want[2][[0, 2]])


def test_nan_of_every_kind_ends(gpu):
    """A gate whose bits are all ones, as the words that workgroups wait for are."""
    c = case([700], 8, F4, gpu, True, seed=6)
    c["gate"].view(torch.int32)[::3] = -1
    h, out = forward(c, gpu)
    assert torch.isnan(h).all() and torch.isnan(out).all()
    gg, _, gin = backward(c, h, gpu)
    assert torch.isnan(gin).all() and torch.isnan(gg).all()


def test_bounds_outside_the_rows_are_clamped(gpu):
    c = case([50], 16, BF, gpu, False, seed=7)
    want, _ = forward(c, gpu)
    c["cu"] = torch.tensor([-5, 1000], device=gpu)
    got, _ = forward(c, gpu)
    assert torch.equal(got, want)


def test_backward_against_differences(gpu):
    lens, d, eps = [20, 7], 16, 1e-3
    c = case(lens, d, F4, gpu, True, seed=8)
    h, _ = forward(c, gpu)
    gg, gu, gin = backward(c, h, gpu)
    g = torch.Generator().manual_seed(1)
    base = {"gate": c["gate"].cpu().double(), "u": c["u"].cpu().double(), "s0": c["s0"].cpu().double()}

    def loss(v):
        (h64, _), (s64, _) = recurrence(v["gate"], v["u"], lens, v["s0"])
        return (h64 * c["gh"].cpu().double()).sum() + (s64 * c["ds"].cpu().double()).sum()
    for name, grad in (("gate", gg), ("u", gu), ("s0", gin)):
        for _ in range(4):
            d_ = torch.randn(grad.shape, generator=g, dtype=torch.float64)
            up, down = ({**base, name: base[name] + s * eps * d_} for s in (1, -1))
            want = (loss(up) - loss(down)) / (2 * eps)
            got = (grad.cpu().double() * d_).sum()
            assert abs(got - want) <= 1e-4 * (grad.cpu().double() * d_).abs().sum(), name


@pytest.mark.parametrize("dtype", [BF, FP, F4], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [8, 512, 2056, 5120])
def test_step(gpu, d, dtype):
    c = case([9], d, dtype, gpu, False, seed=9, apart=True)
    g = torch.Generator().manual_seed(2)
    pool = torch.randn((6, d), generator=g).to(gpu)
    slots = torch.tensor([4, -1, 2, 0, 6, 2, 1 << 40, 2, 5], device=gpu)  # slot 2: three tokens of one sequence
    state = pool.clone()
    h, whole = poisoned((9, d), dtype, gpu, d + 16)
    eg.engram_gated_scan_step(c["gate"], c["u"], state, slots, h)
    torch.cuda.synchronize()
    assert around_untouched(whole, d)
    for slot, rows in ((4, [0]), (2, [2, 5, 7]), (0, [3]), (5, [8])):
        (h64, eh), (s64, es) = recurrence(c["gate"][rows], c["u"][rows], [len(rows)], pool[slot:slot + 1])
        check("h", h[rows], h64, eh + rounded(h64, dtype))
        check("state", state[slot], s64[0], es[0] + F32 * s64[0].abs())
    assert torch.isnan(h[[1, 4, 6]]).all() and torch.equal(state[[1, 3]], pool[[1, 3]])


def test_steps_go_on_where_a_prompt_ended(gpu):
    c = case([130, 70], 520, BF, gpu, True, seed=10)
    h, _ = forward(c, gpu)
    short = {**c, "lens": [120, 60], "cu": torch.tensor([0, 120, 180], device=gpu), "n": 180, "b": 2}
    cut = torch.cat((torch.arange(120), torch.arange(130, 190))).to(gpu)
    short["gate"], short["u"] = c["gate"][cut], c["u"][cut]
    _, state = forward(short, gpu)
    slots, row = torch.tensor([0, 1], device=gpu), torch.empty((2, 520), dtype=BF, device=gpu)
    for i in range(10):
        at = torch.tensor([120 + i, 190 + i], device=gpu)
        eg.engram_gated_scan_step(c["gate"][at], c["u"][at], state, slots, row)
        # both round states that differ in fp32's last digits: at most a step of bf16 (2^-7) apart
        assert ((row.double() - h[at].double()).abs() <= 2.0 ** -7 * h[at].double().abs() + 1e-6).all()


def test_captured_and_replayed_and_two_streams(gpu):
    c = case([900, 333], 1368, BF, gpu, True, seed=11)
    n, b, d = c["n"], c["b"], c["d"]
    need = eg.engram_gated_scan_fwd_workspace_bytes(n, b, d)

    def buffers():
        t = torch.empty
        return [t((n, d), dtype=BF, device=gpu), t((b, d), device=gpu), t((n, d), dtype=BF, device=gpu),
                t((n, d), dtype=BF, device=gpu), t((b, d), device=gpu), t(need, dtype=torch.uint8, device=gpu)]

    def step(h, out, gg, gu, gin, ws):
        eg.engram_gated_scan_fwd(c["gate"], c["u"], c["cu"], h, ws, state_in=c["s0"], state_out=out)
        eg.engram_gated_scan_bwd(c["gh"], c["gate"], c["u"], h, c["cu"], gg, gu, ws, state_in=c["s0"],
                                 grad_state_out=c["ds"], grad_state_in=gin)
    want, other, kept = buffers(), buffers(), buffers()
    step(*want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = buffers()
    for _ in range(3):
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
