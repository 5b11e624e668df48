"""Rows so far apart that the last ones lie behind 2^32 values, and a state pool
of more than 2^32 bytes: bit for bit what the same rows side by side give."""
from __future__ import annotations

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import poisoned

pytestmark = pytest.mark.gpu
BF, F4 = torch.bfloat16, torch.float32
LD, N = 1048576, 4200  # 4.4e9 values from the first row to the last


@pytest.fixture(scope="module")
def space(gpu):
    """Room for rows that far apart, 8.8 GB; its contents are whatever they are."""
    t = torch.empty(LD * N, dtype=BF, device=gpu)
    yield t
    del t
    torch.cuda.empty_cache()


def far(space, at, t):
    """t's rows as columns `at` .. of the far rows."""
    width = t[0].numel()
    v = torch.as_strided(space, (N, width), (LD, 1), at)
    v.copy_(t.reshape(N, width))
    return v.unflatten(1, tuple(t.shape[1:])) if t.dim() > 2 else v


def same(name, a, b):
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), name


def ws(need, dev):
    return poisoned((max(need, 16),), torch.uint8, dev)


def test_linear(gpu, space):
    k, m = 136, 72
    g = torch.Generator(device=gpu).manual_seed(1)
    x, w = torch.randn((N, k), generator=g, device=gpu).to(BF), torch.randn((m, k), generator=g, device=gpu).to(BF)
    gy, res = (torch.randn((N, m), generator=g, device=gpu).to(BF) for _ in range(2))
    out = []
    for apart in (False, True):
        p = {"x": x, "gy": gy, "res": res, "y": poisoned((N, m), BF, gpu), "z": poisoned((N, m), BF, gpu),
             "gx": poisoned((N, k), BF, gpu)}
        if apart:
            p = {s: far(space, 1024 * (i + 1), t) for i, (s, t) in enumerate(p.items())}
        gw, gb = poisoned((m, k), BF, gpu), poisoned((m,), F4, gpu)
        eg.engram_linear_fwd(p["x"], w, p["y"], ws(eg.engram_linear_fwd_workspace_bytes(N, k, m), gpu), residual=p["res"],
                             z=p["z"], act="silu")
        eg.engram_linear_bwd(p["gy"], p["x"], w, p["gx"], gw, ws(eg.engram_linear_bwd_workspace_bytes(N, k, m), gpu),
                             z=p["z"], grad_bias=gb, act="silu")
        torch.cuda.synchronize()
        out.append({"y": p["y"].clone(), "z": p["z"].clone(), "gx": p["gx"].clone(), "gw": gw, "gb": gb})
    for s in out[0]:
        same(s, out[0][s], out[1][s])


def test_norms(gpu, space):
    hq, hk, d, r = 3, 2, 72, 48
    g = torch.Generator(device=gpu).manual_seed(2)

    def rand(*s):
        return torch.randn(s, generator=g, device=gpu)
    wq, wk, freqs = rand(d), rand(d), eg.engram_rope_freqs(10000.0, r).to(gpu)
    pos = torch.arange(N, device=gpu) * 1000003
    q, k, gq, gk = rand(N, hq, d).to(BF), rand(N, hk, d).to(BF), rand(N, hq, d).to(BF), rand(N, hk, d).to(BF)
    out = []
    for apart in (False, True):
        p = {"q": q, "k": k, "gqo": gq, "gko": gk}
        p.update({s: poisoned((N, h, d), BF, gpu) for s, h in (("qo", hq), ("ko", hk), ("gq", hq), ("gk", hk))})
        if apart:
            p = {s: far(space, 1024 * (i + 1), t) for i, (s, t) in enumerate(p.items())}
        gwq, gwk = poisoned((d,), F4, gpu), poisoned((d,), F4, gpu)
        eg.engram_qk_norm_rope_fwd(p["q"], p["k"], wq, wk, pos, freqs, p["qo"], p["ko"])
        eg.engram_qk_norm_rope_bwd(p["gqo"], p["gko"], p["q"], p["k"], wq, wk, pos, freqs, p["gq"], p["gk"], gwq, gwk,
                                   ws(eg.engram_qk_norm_rope_bwd_workspace_bytes(N, hq, hk, d), gpu))
        torch.cuda.synchronize()
        out.append({**{s: p[s].clone() for s in ("qo", "ko", "gq", "gk")}, "gwq": gwq, "gwk": gwk})
    for s in out[0]:
        same(s, out[0][s], out[1][s])


def test_decay(gpu, space):
    h, dk, dv, lens = 2, 40, 72, [3000, 0, 1150]
    g = torch.Generator(device=gpu).manual_seed(3)

    def rand(*s):
        return torch.randn(s, generator=g, device=gpu)
    ld = torch.tensor([-0.01, -0.3], device=gpu)
    cu = torch.tensor([0] + lens).cumsum(0).to(gpu)
    q, k, v, do = (rand(N, h, d).to(BF) for d in (dk, dk, dv, dv))
    s0, ds = rand(3, h, dk, dv), rand(3, h, dk, dv)
    out = []
    for apart in (False, True):
        p = {"q": q, "k": k, "v": v, "do": do, "o": poisoned((N, h, dv), BF, gpu)}
        p.update({s: poisoned((N, h, d), BF, gpu) for s, d in (("gq", dk), ("gk", dk), ("gv", dv))})
        if apart:
            p = {s: far(space, 1024 * (i + 1), t) for i, (s, t) in enumerate(p.items())}
        s1, gs = poisoned((3, h, dk, dv), F4, gpu), poisoned((3, h, dk, dv), F4, gpu)
        eg.engram_decay_attn_fwd(p["q"], p["k"], p["v"], ld, cu, p["o"],
                                 ws(eg.engram_decay_attn_fwd_workspace_bytes(N, 3, h, dk, dv), gpu), scale=0.2, state_in=s0,
                                 state_out=s1)
        eg.engram_decay_attn_bwd(p["do"], p["q"], p["k"], p["v"], ld, cu, p["gq"], p["gk"], p["gv"],
                                 ws(eg.engram_decay_attn_bwd_workspace_bytes(N, 3, h, dk, dv), gpu), scale=0.2, state_in=s0,
                                 grad_state_out=ds, grad_state_in=gs)
        torch.cuda.synchronize()
        out.append({**{s: p[s].clone() for s in ("o", "gq", "gk", "gv")}, "s1": s1, "gs": gs})
    for s in out[0]:
        same(s, out[0][s], out[1][s])
    assert torch.isnan(out[1]["o"][4150:]).all()


def test_a_pool_of_states_beyond_32_bits(gpu):
    h, d, slots = 4, 128, 20000  # 5.2 GB
    g = torch.Generator(device=gpu).manual_seed(4)

    def rand(*s):
        return torch.randn(s, generator=g, device=gpu)
    pool = torch.empty((slots, h, d, d), device=gpu)
    places = torch.tensor([slots - 1, 0, 16384, slots - 2], device=gpu)
    state = rand(4, h, d, d)
    pool[places] = state
    q, k, v, ld = rand(4, h, d).to(BF), rand(4, h, d).to(BF), rand(4, h, d).to(BF), -rand(h).abs()
    o, o2 = poisoned((4, h, d), BF, gpu), poisoned((4, h, d), BF, gpu)
    eg.engram_decay_attn_step(q, k, v, ld, pool, places, o, scale=0.1)
    eg.engram_decay_attn_step(q, k, v, ld, state, torch.arange(4, device=gpu), o2, scale=0.1)
    torch.cuda.synchronize()
    same("o", o, o2)
    same("state", pool[places], state)
