"""The decay attention on the GPU against its recurrence in 64 bits: ragged and
empty sequences, carried states, head sizes, decays from none to total, rows
behind the last sequence, infinities; the backward against the reversed
recurrence and against differences; the step against the recurrence."""
from __future__ import annotations

import math

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import F32, around_untouched, check, poisoned, rounded

pytestmark = pytest.mark.gpu
BF, F4 = torch.bfloat16, torch.float32
U = 2.0 ** -8          # half a step of bf16
SPLIT = 2.0 ** -16     # a value as the sum of two bf16
POWER = 2.0 ** -17     # a power of the decay in fp32: |log lam| steps is off by 2^-24 of itself, and below 88 where it matters


def recurrence(q, k, v, ld, lens, scale, s0):
    """o and final states, in 64 bits on the CPU (or wherever the inputs are)."""
    n, h, dk = q.shape
    dv = v.shape[2]
    lam = torch.exp(ld.double())[:, None, None]
    o = torch.zeros((n, h, dv), dtype=torch.float64, device=q.device)
    out = torch.zeros((len(lens), h, dk, dv), dtype=torch.float64, device=q.device)
    at = 0
    for b, length in enumerate(lens):
        s = torch.zeros((h, dk, dv), dtype=torch.float64, device=q.device) if s0 is None else s0[b].double()
        for t in range(at, at + length):
            s = lam * s + k[t].double()[:, :, None] * v[t].double()[:, None, :]
            o[t] = scale * (q[t].double()[:, :, None] * s).sum(1)
        at += length
        out[b] = s
    return o, out


def reversed_recurrence(do, q, k, v, ld, lens, scale, s0, ds):
    n, h, dk = q.shape
    dv = v.shape[2]
    lam = torch.exp(ld.double())[:, None, None]
    do, q, k, v = (x.double() for x in (do, q, k, v))
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    din = torch.zeros((len(lens), h, dk, dv), dtype=torch.float64, device=q.device)
    at = 0
    for b, length in enumerate(lens):
        s = torch.zeros((h, dk, dv), dtype=torch.float64, device=q.device) if s0 is None else s0[b].double()
        g = torch.zeros((h, dk, dv), dtype=torch.float64, device=q.device) if ds is None else ds[b].double()
        for t in range(at, at + length):
            s = lam * s + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * (s * do[t][:, None, :]).sum(2)
        for t in reversed(range(at, at + length)):
            g = g + scale * q[t][:, :, None] * do[t][:, None, :]
            dkk[t] = (g * v[t][:, None, :]).sum(2)
            dvv[t] = (g * k[t][:, :, None]).sum(1)
            g = lam * g
        at += length
        din[b] = g
    return dq, dkk, dvv, din


def case(lens, h, dk, dv, dev, states, tail=0, seed=0, ld=None, apart=False):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens) + tail

    def r(*s):
        return torch.randn(s, generator=g)
    if apart:
        packed = r(n, h * (2 * dk + dv) + 16).to(BF).to(dev)
        q, k = packed[:, :h * dk].unflatten(1, (h, dk)), packed[:, h * dk:2 * h * dk].unflatten(1, (h, dk))
        v = packed[:, 2 * h * dk:h * (2 * dk + dv)].unflatten(1, (h, dv))
    else:
        q, k, v = r(n, h, dk).to(BF).to(dev), r(n, h, dk).to(BF).to(dev), r(n, h, dv).to(BF).to(dev)
    b = len(lens)
    if ld is None:
        ld = -torch.pow(2.0, -torch.arange(h, dtype=torch.float32) * 7 / max(1, h) - 1)
    c = {"q": q, "k": k, "v": v, "do": r(n, h, dv).to(BF).to(dev), "ld": ld.to(dev), "scale": dk ** -0.5,
         "cu": torch.tensor([0] + lens).cumsum(0).to(dev), "lens": lens, "n": n, "h": h, "dk": dk, "dv": dv,
         "s0": r(b, h, dk, dv).to(dev) if states else None, "ds": r(b, h, dk, dv).to(dev) if states else None}
    return c


def cpu(c, *names):
    return [None if c[s] is None else c[s].cpu() for s in names]


def run_fwd(c, dev, state_out=True, ldo=None, stream=None):
    n, b, h, dk, dv = c["n"], len(c["lens"]), c["h"], c["dk"], c["dv"]
    o, whole = poisoned((n, h, dv), BF, dev, ldo or h * dv + 8)
    out = poisoned((b, h, dk, dv), F4, dev) if state_out else None
    ws = poisoned((eg.engram_decay_attn_fwd_workspace_bytes(n, b, h, dk, dv),), torch.uint8, dev)
    eg.engram_decay_attn_fwd(c["q"], c["k"], c["v"], c["ld"], c["cu"], o, ws, scale=c["scale"], state_in=c["s0"],
                             state_out=out, stream=stream)
    torch.cuda.synchronize()
    assert around_untouched(whole, h * dv)
    return o, out


def fwd_bounds(c):
    """The recurrence, and the same over absolute values, which bounds every sum of absolute products."""
    q, k, v, ld, s0 = cpu(c, "q", "k", "v", "ld", "s0")
    m = sum(c["lens"])
    o, s = recurrence(q[:m], k[:m], v[:m], ld, c["lens"], c["scale"], s0)
    oa, sa = recurrence(q[:m].abs(), k[:m].abs(), v[:m].abs(), ld, c["lens"], c["scale"], None if s0 is None else s0.abs())
    # X is scaled and added to once a chunk: 64 + 8 fp32 additions a chunk (the oldest chunk's share sees all)
    steps = F32 * 72 * (max(c["lens"]) / 64 + 2)
    serr = (SPLIT + POWER + steps) * sa
    # scores and X are each rounded once, then the fp32 sums over Dk and 64 rows
    oerr = rounded(o, BF) + (1 + U) * (U * (1 + U) + POWER + steps + SPLIT + F32 * (c["dk"] + 80)) * oa
    return (o, oerr), (s, serr + 1e-37)


LENS = [[1], [63], [64], [65], [200], [1, 0, 3, 64, 129, 0, 2], [0, 0, 5], [128, 128], [700]]
DIMS = [(128, 128), (64, 64), (32, 96), (8, 8), (72, 128), (128, 40)]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dk,dv", DIMS)
def test_forward(gpu, lens, dk, dv):
    for states in (False, True):
        print(f"decay fwd lens={lens} dk={dk} dv={dv} states={states}", flush=True)
        c = case(lens, 3, dk, dv, gpu, states, tail=5, apart=states)
        o, out = run_fwd(c, gpu)
        m = sum(lens)
        (o64, oerr), (s64, serr) = fwd_bounds(c)
        check("o", o[:m], o64.to(gpu), oerr.to(gpu))
        check("state_out", out, s64.to(gpu), serr.to(gpu))
        assert torch.isnan(o[m:]).all()  # rows behind the last sequence: left as they were
        o2, _ = run_fwd(c, gpu, state_out=False)
        assert torch.equal(o[:m], o2[:m])


@pytest.mark.parametrize("ld", [0.0, -1e-6, -3.0, -60.0, -math.inf])
def test_decays_from_none_to_total(gpu, ld):
    c = case([150, 70], 2, 64, 128, gpu, True, ld=torch.tensor([ld, -0.1]), seed=3)
    o, out = run_fwd(c, gpu)
    (o64, oerr), (s64, serr) = fwd_bounds(c)
    check("o", o, o64.to(gpu), oerr.to(gpu))
    check("state_out", out, s64.to(gpu), serr.to(gpu))
    grads = run_bwd(c, gpu)
    for name, got, (want, bound) in zip(("dq", "dk", "dv", "ds_in"), grads, bwd_bounds(c)):
        check(name, got, want.to(gpu), bound.to(gpu))


def run_bwd(c, dev, apart=False, stream=None):
    n, b, h, dk, dv = c["n"], len(c["lens"]), c["h"], c["dk"], c["dv"]
    pad = 16 if apart else 8
    (gq, _), (gk, _), (gv, _) = (poisoned((n, h, d), BF, dev, h * d + pad) for d in (dk, dk, dv))
    gin = poisoned((b, h, dk, dv), F4, dev) if c["s0"] is not None else None
    ws = poisoned((eg.engram_decay_attn_bwd_workspace_bytes(n, b, h, dk, dv),), torch.uint8, dev)
    eg.engram_decay_attn_bwd(c["do"], c["q"], c["k"], c["v"], c["ld"], c["cu"], gq, gk, gv, ws, scale=c["scale"],
                             state_in=c["s0"], grad_state_out=c["ds"], grad_state_in=gin, stream=stream)
    torch.cuda.synchronize()
    return gq, gk, gv, gin


def bwd_bounds(c):
    do, q, k, v, ld, s0, ds = cpu(c, "do", "q", "k", "v", "ld", "s0", "ds")
    m = sum(c["lens"])
    args = [x[:m] for x in (do, q, k, v)]
    want = reversed_recurrence(*args, ld, c["lens"], c["scale"], s0, ds)
    size = reversed_recurrence(*(x.abs() for x in args), ld, c["lens"], c["scale"], None if s0 is None else s0.abs(),
                               None if ds is None else ds.abs())
    steps = F32 * 72 * (max(c["lens"]) / 64 + 2)
    out = []
    for i, (w, a) in enumerate(zip(want, size)):
        if i < 3:
            out.append((w, rounded(w, BF) + (1 + U) * (U * (1 + U) + POWER + steps + SPLIT + F32 * (max(c["dk"], c["dv"]) + 80)) * a))
        else:
            out.append((w, (SPLIT + POWER + steps) * a + 1e-37))
    return out


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dk,dv", DIMS)
def test_backward(gpu, lens, dk, dv):
    for states in (False, True):
        print(f"decay bwd lens={lens} dk={dk} dv={dv} states={states}", flush=True)
        c = case(lens, 3, dk, dv, gpu, states, tail=5, apart=states, seed=1)
        got = run_bwd(c, gpu)
        m = sum(lens)
        for i, (name, g, (want, bound)) in enumerate(zip(("dq", "dk", "dv", "ds_in"), got, bwd_bounds(c))):
            if g is None:
                continue
            check(name, g[:m] if i < 3 else g, want.to(gpu), bound.to(gpu))
            if i < 3:
                assert torch.isnan(g[m:]).all()


def test_backward_against_differences(gpu):
    """<gradient, direction> against differences of the 64-bit recurrence, L = <o, do> + <state_out, ds>."""
    c = case([70, 9], 2, 32, 40, gpu, True, seed=2)
    grads = run_bwd(c, gpu)
    bounds = bwd_bounds(c)
    do, q, k, v, ld, s0, ds = cpu(c, "do", "q", "k", "v", "ld", "s0", "ds")
    base = {"q": q.double(), "k": k.double(), "v": v.double(), "s0": s0.double()}
    gen = torch.Generator().manual_seed(4)
    for name, got, (_, bound) in zip(("q", "k", "v", "s0"), grads, bounds):
        u = torch.randn(base[name].shape, generator=gen, dtype=torch.float64)

        def loss(t):
            a = {s: x + (t * u if s == name else 0) for s, x in base.items()}
            o, s = recurrence(a["q"], a["k"], a["v"], ld, c["lens"], c["scale"], a["s0"])
            return ((o * do.double()).sum() + (s * ds.double()).sum()).item()
        h = 1e-4  # the loss is linear in each of the four, so only its rounding is left
        want = (loss(h) - loss(-h)) / (2 * h)
        have = (got.double().cpu() * u).sum().item()
        assert abs(have - want) <= (bound * u.abs()).sum().item() + 1e-6 * abs(want), (name, have, want)


def test_a_sequence_in_pieces(gpu):
    """Carrying state_out into the next call's state_in continues the sequence."""
    c = case([300], 2, 64, 64, gpu, True, seed=5)
    (o64, oerr), (s64, serr) = fwd_bounds(c)
    state, outs = c["s0"], []
    for lo, hi in ((0, 1), (1, 100), (100, 228), (228, 300)):
        p = dict(c, q=c["q"][lo:hi], k=c["k"][lo:hi], v=c["v"][lo:hi], n=hi - lo, lens=[hi - lo], s0=state,
                 cu=torch.tensor([0, hi - lo], device=gpu))
        o, state = run_fwd(p, gpu)
        outs.append(o)
    check("o", torch.cat(outs), o64.to(gpu), 2 * oerr.to(gpu))
    check("state", state, s64.to(gpu), 2 * serr.to(gpu))


def test_many_sequences(gpu):
    """More sequences than fit beside each other, most of them tiny, some empty."""
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(0, 4, (700,), generator=g).tolist()
    lens[300] = 400
    c = case(lens, 1, 16, 24, gpu, True, seed=6)
    o, out = run_fwd(c, gpu)
    (o64, oerr), (s64, serr) = fwd_bounds(c)
    check("o", o, o64.to(gpu), oerr.to(gpu))
    check("state_out", out, s64.to(gpu), serr.to(gpu))


@pytest.mark.parametrize("bad", [math.inf, math.nan, -math.inf])
def test_later_rows_and_other_sequences_do_not_reach_back(gpu, bad):
    """A value that is not finite in a token's q, k or v changes nothing before it in its
    sequence, nothing in the other sequences and heads, bit for bit outside its own chunk
    and within the bounds inside it."""
    c = case([150, 90], 2, 64, 64, gpu, False, seed=7)
    clean, sclean = run_fwd(c, gpu)
    (o64, oerr), _ = fwd_bounds(c)
    for what in "qkv":
        x = {s: c[s].clone() for s in "qkv"}
        x[what][100, 1, 3] = bad
        o, s = run_fwd(dict(c, **x), gpu)
        check("before", o[:100], o64[:100].to(gpu), oerr[:100].to(gpu))
        assert torch.equal(o[150:].view(torch.int16), clean[150:].view(torch.int16))
        assert torch.equal(o[:64].view(torch.int16), clean[:64].view(torch.int16))
        assert torch.equal(o[:, 0].view(torch.int16), clean[:, 0].view(torch.int16))
        assert torch.equal(s[1], sclean[1])
        assert not torch.isfinite(o[100, 1]).all()
        if what == "q":  # a query's rows are its own
            keep = [i for i in range(240) if i != 100]
            assert torch.equal(o[keep].view(torch.int16), clean[keep].view(torch.int16))


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_gradients_do_not_reach_forward(gpu, bad):
    """The same of the backward: what is not finite at a token t reaches dq from t on (through k
    and v) and dk and dv up to t (through q and grad_o), in its own sequence and head."""
    lens, t = [150, 90], 100
    c = case(lens, 2, 64, 64, gpu, False, seed=11)
    clean = run_bwd(c, gpu)[:3]
    bounds = bwd_bounds(c)[:3]
    for what in ("do", "q", "k", "v"):
        x = c[what].clone()
        x[t, 1, 3] = bad
        got = run_bwd(dict(c, **{what: x}), gpu)[:3]
        for i, (name, g, keep) in enumerate(zip(("dq", "dk", "dv"), got, clean)):
            assert torch.equal(g[:, 0].view(torch.int16), keep[:, 0].view(torch.int16)), (what, name)
            assert torch.equal(g[150:].view(torch.int16), keep[150:].view(torch.int16)), (what, name)
            rows = torch.ones(150, dtype=torch.bool)
            reached = what in ("k", "v") if name == "dq" else what in ("q", "do")
            if reached:
                rows[(slice(t, None) if name == "dq" else slice(0, t + 1))] = False
            rows[t] = False
            want, bound = bounds[i]
            check(f"{name} with {what}", g[:150][rows.to(gpu)], want[:150][rows].to(gpu), bound[:150][rows].to(gpu))


@pytest.mark.parametrize("lens,h,dk,dv", [([70, 3], 600, 8, 8), ([900, 500], 40, 16, 24), ([400], 200, 72, 8)])
def test_heads_that_fill_the_chip(gpu, lens, h, dk, dv):
    """Many heads: the axis in few segments of many chunks each, or in one; other numbers of
    them forward and backward."""
    print(f"decay lens={lens} h={h} dk={dk} dv={dv}", flush=True)
    c = case(lens, h, dk, dv, gpu, True, tail=2, seed=12)
    m = sum(lens)
    o, out = run_fwd(c, gpu)
    (o64, oerr), (s64, serr) = fwd_bounds(c)
    check("o", o[:m], o64.to(gpu), oerr.to(gpu))
    check("state_out", out, s64.to(gpu), serr.to(gpu))
    for i, (name, g, (want, bound)) in enumerate(zip(("dq", "dk", "dv", "ds_in"), run_bwd(c, gpu), bwd_bounds(c))):
        check(name, g[:m] if i < 3 else g, want.to(gpu), bound.to(gpu))


def test_bounds_of_sequences_that_lead_nowhere(gpu):
    """cu_seqlens of any content leads to no access outside the arrays: the call ends, and
    what belongs to nobody else is not written."""
    c = case([40, 40], 2, 64, 64, gpu, True, seed=8)
    for cu in ([0, 300, 80], [-5, 40, 1 << 40], [80, 40, 0], [0, 0, 0]):
        o, out = run_fwd(dict(c, cu=torch.tensor(cu, device=gpu)), gpu)
        run_bwd(dict(c, cu=torch.tensor(cu, device=gpu)), gpu)
    assert torch.isnan(o).all()  # no sequence has a row
    assert torch.equal(out, c["s0"])


# ---------------------------------------------------------------- the step


def step_case(b, h, dk, dv, pool, dev, seed=0, apart=False):
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g)
    packed = r(b, h * (2 * dk + dv) + (24 if apart else 0)).to(BF).to(dev)
    c = {"q": packed[:, :h * dk].unflatten(1, (h, dk)), "k": packed[:, h * dk:2 * h * dk].unflatten(1, (h, dk)),
         "v": packed[:, 2 * h * dk:h * (2 * dk + dv)].unflatten(1, (h, dv)), "state": r(pool, h, dk, dv).to(dev),
         "ld": (-torch.rand((h,), generator=g)).to(dev), "scale": dk ** -0.5}
    return c


def step64(c, slots):
    q, k, v, ld = (c[s].cpu().double() for s in ("q", "k", "v", "ld"))
    st, sa = c["state"].cpu().double(), c["state"].cpu().double().abs()
    lam = torch.exp(ld)[:, None, None]
    o, oa = (torch.zeros(v.shape, dtype=torch.float64) for _ in range(2))
    for i, s in enumerate(slots):
        if 0 <= s < st.shape[0]:
            st[s] = lam * st[s] + k[i][:, :, None] * v[i][:, None, :]
            sa[s] = lam * sa[s] + (k[i][:, :, None] * v[i][:, None, :]).abs()
            o[i] = c["scale"] * (q[i][:, :, None] * st[s]).sum(1)
            oa[i] = c["scale"] * (q[i].abs()[:, :, None] * sa[s]).sum(1)
    return o, oa, st, sa


STEPS = [(1, 40, 128, 128, [3]), (2, 3, 8, 8, [1, 0]), (5, 2, 64, 128, [4, 0, 2, 9, 1]), (7, 3, 72, 40, [0, 1, -1, 3, 100, 5, 6]),
         (6, 2, 128, 64, [2, 2, 5, 2, 5, 0]), (16, 40, 128, 128, list(range(15, -1, -1))), (300, 2, 32, 24, [i % 7 for i in range(300)])]


@pytest.mark.parametrize("b,h,dk,dv,slots", STEPS)
@pytest.mark.parametrize("apart", [False, True])
def test_step(gpu, b, h, dk, dv, slots, apart):
    print(f"decay step b={b} h={h} dk={dk} dv={dv} apart={apart}", flush=True)
    pool = 10 if b < 16 else 20
    c = step_case(b, h, dk, dv, pool, gpu, seed=b, apart=apart)
    o64, oa, s64, sa = step64(c, slots)
    o, whole = poisoned((b, h, dv), BF, gpu, h * dv + 8)
    eg.engram_decay_attn_step(c["q"], c["k"], c["v"], c["ld"], c["state"], torch.tensor(slots, device=gpu), o,
                              scale=c["scale"])
    torch.cuda.synchronize()
    times = max(slots.count(s) for s in slots) + 1
    serr = F32 * 4 * times * sa + 1e-37
    oerr = rounded(o64, BF) + (1 + U) * F32 * (dk + 4 + 4 * times) * oa
    used = torch.tensor([0 <= s < pool for s in slots])
    check("o", o[used.to(gpu)], o64[used].to(gpu), oerr[used].to(gpu))
    check("state", c["state"], s64.to(gpu), serr.to(gpu))
    assert torch.isnan(o[~used.to(gpu)]).all() and around_untouched(whole, h * dv)


def test_steps_continue_a_prompt(gpu):
    """A prompt through the forward, then tokens one by one: the recurrence over all of them."""
    h, d, t, more = 2, 64, 70, 5
    c = case([t + more], h, d, d, gpu, True, seed=9)
    (o64, oerr), (s64, serr) = fwd_bounds(c)
    p = dict(c, q=c["q"][:t], k=c["k"][:t], v=c["v"][:t], n=t, lens=[t], cu=torch.tensor([0, t], device=gpu))
    _, state = run_fwd(p, gpu)
    slots = torch.zeros(1, dtype=torch.int64, device=gpu)
    for i in range(t, t + more):
        o = poisoned((1, h, d), BF, gpu)
        eg.engram_decay_attn_step(c["q"][i:i + 1], c["k"][i:i + 1], c["v"][i:i + 1], c["ld"], state, slots, o, scale=c["scale"])
        torch.cuda.synchronize()
        check("o", o[0], o64[i].to(gpu), oerr[i].to(gpu))
    check("state", state, s64.to(gpu), 2 * serr.to(gpu))


def test_graph_and_streams(gpu):
    """All three calls captured and replayed with eager work between, and forward and
    backward on two other streams at once: bit for bit the eager results."""
    c = case([200, 3, 90], 4, 64, 64, gpu, True, seed=10)
    want_f, want_b = run_fwd(c, gpu), run_bwd(c, gpu)
    s = step_case(6, 4, 64, 64, 8, gpu, seed=11)
    slots = torch.tensor([1, 5, 2, 0, 2, -1], device=gpu)
    n, b, h, d = c["n"], 3, 4, 64
    ws = [poisoned((eg.engram_decay_attn_bwd_workspace_bytes(n, b, h, d, d),), torch.uint8, gpu) for _ in range(4)]

    def buffers():
        return [poisoned((n, h, d), BF, gpu) for _ in range(4)], [poisoned((b, h, d, d), F4, gpu) for _ in range(2)]

    def go(bufs, wf, wb, stream=None):
        (o, gq, gk, gv), (out, gin) = bufs
        eg.engram_decay_attn_fwd(c["q"], c["k"], c["v"], c["ld"], c["cu"], o, wf, scale=c["scale"], state_in=c["s0"],
                                 state_out=out, stream=stream)
        eg.engram_decay_attn_bwd(c["do"], c["q"], c["k"], c["v"], c["ld"], c["cu"], gq, gk, gv, wb, scale=c["scale"],
                                 state_in=c["s0"], grad_state_out=c["ds"], grad_state_in=gin, stream=stream)

    def same(bufs):
        (o, gq, gk, gv), (out, gin) = bufs
        pairs = [(o, want_f[0]), (out, want_f[1]), (gq, want_b[0]), (gk, want_b[1]), (gv, want_b[2]), (gin, want_b[3])]
        return all(torch.equal(x, y) for x, y in pairs)
    bufs = buffers()
    first = s["state"].clone()
    so = poisoned((6, 4, 64), BF, gpu)

    def step(state, o):
        eg.engram_decay_attn_step(s["q"], s["k"], s["v"], s["ld"], state, slots, o, scale=s["scale"])
    eager_state, eager_o = first.clone(), poisoned((6, 4, 64), BF, gpu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(bufs, ws[0], ws[1])
        step(s["state"], so)
    for _ in range(3):
        for t in bufs[0] + bufs[1] + ws[:2]:
            t.view(torch.uint8).fill_(0xFF)
        torch.randn(1000, device=gpu).sum().item()
        graph.replay()
        step(eager_state, eager_o)
        torch.cuda.synchronize()
        assert same(bufs)
        assert torch.equal(s["state"], eager_state) and torch.equal(so[:5], eager_o[:5])
    streams, sets = [torch.cuda.Stream() for _ in range(2)], [buffers(), buffers()]
    torch.cuda.synchronize()
    for i, (st, o) in enumerate(zip(streams, sets)):
        go(o, ws[2 * i], ws[2 * i + 1], stream=st)
    torch.cuda.synchronize()
    assert same(sets[0]) and same(sets[1])
