"""Rows so far apart that the last ones lie behind 2^32 values, and pools of caches
and states of more than 2^32 bytes: bit for bit what the same gives side by side."""
from __future__ import annotations

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import poisoned
from test_gpu_layers_far import N, far, same, space, ws  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
BF, F4 = torch.bfloat16, torch.float32


def normal(dev, *shape, seed):
    return torch.randn(shape, generator=torch.Generator(device=dev).manual_seed(seed), device=dev).to(BF)


def both(space, names, call):
    """`call` over the tensors as they are and over far rows."""
    out = []
    for apart in (False, True):
        p = {s: far(space, 1024 * (i + 1), t) if apart else t.clone() for i, (s, t) in enumerate(names.items())}
        rest = call(p)
        torch.cuda.synchronize()
        out.append({**{s: t.clone() for s, t in p.items()}, **rest})
    for s in out[0]:
        same(s, out[0][s], out[1][s])


def test_layer_norm(gpu, space):  # noqa: F811
    d = 520
    w = normal(gpu, d, seed=1).float()

    def call(p):
        saved, gw, gb = poisoned((N, 2), F4, gpu), poisoned((d,), F4, gpu), poisoned((d,), F4, gpu)
        eg.engram_layer_norm_fwd(p["x"], w, p["y"], saved=saved)
        eg.engram_layer_norm_bwd(p["gy"], p["x"], w, saved, p["gx"], ws(eg.engram_layer_norm_bwd_workspace_bytes(N, d), gpu),
                                 grad_w=gw, grad_b=gb, grad_residual=p["r"])
        return {"saved": saved, "gw": gw, "gb": gb}
    blank = poisoned((N, d), BF, gpu)
    both(space, {"x": normal(gpu, N, d, seed=2), "gy": normal(gpu, N, d, seed=3), "r": normal(gpu, N, d, seed=4), "y": blank,
                 "gx": blank}, call)


def test_window_attention(gpu, space):  # noqa: F811
    hq, hk, d = 4, 2, 72
    cu = torch.tensor([0, 3000, N - 5], device=gpu)

    def call(p):
        lse = poisoned((N, hq), F4, gpu)
        eg.engram_window_attn_fwd(p["q"], p["k"], p["v"], cu, p["o"], 300, sinks=5, lse=lse, scale=0.1)
        eg.engram_window_attn_bwd(p["go"], p["q"], p["k"], p["v"], p["o"], lse, cu, p["gq"], p["gk"], p["gv"],
                                  ws(eg.engram_window_attn_bwd_workspace_bytes(N, 2, hq, hk, d, 300, 5), gpu), 300, sinks=5,
                                  scale=0.1)
        return {"lse": lse}
    q, k = (N, hq, d), (N, hk, d)
    blank_q, blank_k = poisoned(q, BF, gpu), poisoned(k, BF, gpu)
    both(space, {"q": normal(gpu, *q, seed=1), "k": normal(gpu, *k, seed=2), "v": normal(gpu, *k, seed=3),
                 "go": normal(gpu, *q, seed=4), "o": blank_q, "gq": blank_q, "gk": blank_k, "gv": blank_k}, call)


@pytest.mark.parametrize("window,sinks,hq,hk,d", [(1 << 40, 0, 2, 2, 64), (2048, 0, 2, 1, 128), (2048, 5, 2, 1, 128),
                                                  (1950, 0, 2, 1, 72), (2500, 70, 2, 2, 40)])
def test_window_attention_over_more_than_four_gigabytes(gpu, space, window, sinks, hq, hk, d):  # noqa: F811
    """Rows that see 2^32 bytes and more of keys and values, from their first to their last."""
    cu = torch.tensor([0, N - 3], device=gpu)

    def call(p):
        lse = poisoned((N, hq), F4, gpu)
        print(f"far window {window} sinks {sinks} d {d}", flush=True)
        eg.engram_window_attn_fwd(p["q"], p["k"], p["v"], cu, p["o"], window, sinks=sinks, lse=lse, scale=0.1)
        eg.engram_window_attn_bwd(p["go"], p["q"], p["k"], p["v"], p["o"], lse, cu, p["gq"], p["gk"], p["gv"],
                                  ws(eg.engram_window_attn_bwd_workspace_bytes(N, 1, hq, hk, d, window, sinks), gpu), window,
                                  sinks=sinks, scale=0.1)
        return {"lse": lse}
    q, k = (N, hq, d), (N, hk, d)
    blank_q, blank_k = poisoned(q, BF, gpu), poisoned(k, BF, gpu)
    both(space, {"q": normal(gpu, *q, seed=1), "k": normal(gpu, *k, seed=2), "v": normal(gpu, *k, seed=3),
                 "go": normal(gpu, *q, seed=4), "o": blank_q, "gq": blank_q, "gk": blank_k, "gv": blank_k}, call)


def test_window_attention_of_values_that_are_not_finite(gpu, space):  # noqa: F811
    hq, hk, d = 4, 2, 72
    cu = torch.tensor([0, 3000, N - 5], device=gpu)
    k, v, go = normal(gpu, N, hk, d, seed=2), normal(gpu, N, hk, d, seed=3), normal(gpu, N, hq, d, seed=4)
    v[[700, 4100], :, 9], go[[1500, 4000], :, 70], k[2500, :, 3] = float("inf"), float("nan"), float("inf")

    def call(p):
        lse = poisoned((N, hq), F4, gpu)
        eg.engram_window_attn_fwd(p["q"], p["k"], p["v"], cu, p["o"], 300, sinks=5, lse=lse, scale=0.1)
        eg.engram_window_attn_bwd(p["go"], p["q"], p["k"], p["v"], p["o"], lse, cu, p["gq"], p["gk"], p["gv"],
                                  ws(eg.engram_window_attn_bwd_workspace_bytes(N, 2, hq, hk, d, 300, 5), gpu), 300, sinks=5,
                                  scale=0.1)
        return {"lse": lse}
    blank_q, blank_k = poisoned((N, hq, d), BF, gpu), poisoned((N, hk, d), BF, gpu)
    both(space, {"q": normal(gpu, N, hq, d, seed=1), "k": k, "v": v, "go": go, "o": blank_q, "gq": blank_q, "gk": blank_k,
                 "gv": blank_k}, call)


def test_gated_scan(gpu, space):  # noqa: F811
    d = 264
    cu = torch.tensor([0, 3000, 3000, N - 5], device=gpu)

    def call(p):
        s, gs = poisoned((3, d), F4, gpu), poisoned((3, d), F4, gpu)
        eg.engram_gated_scan_fwd(p["gate"], p["u"], cu, p["h"], ws(eg.engram_gated_scan_fwd_workspace_bytes(N, 3, d), gpu),
                                 state_out=s)
        eg.engram_gated_scan_bwd(p["gh"], p["gate"], p["u"], p["h"], cu, p["gg"], p["gu"],
                                 ws(eg.engram_gated_scan_bwd_workspace_bytes(N, 3, d), gpu), grad_state_in=gs)
        return {"s": s, "gs": gs}
    blank = poisoned((N, d), BF, gpu)
    both(space, {"gate": normal(gpu, N, d, seed=1), "u": normal(gpu, N, d, seed=2), "gh": normal(gpu, N, d, seed=3),
                 "h": blank, "gg": blank, "gu": blank}, call)


def test_pool_of_caches(gpu):
    """Five slots of 2^20 lines of two heads of 128: 2.7 GB each for keys and values, and a list of a million tokens."""
    hq, hk, d, lines, sinks = 4, 2, 128, 1 << 20, 4
    pool = 5
    ck, cv = (torch.empty((pool, hk, lines, d), dtype=BF, device=gpu) for _ in range(2))
    small_k, small_v = normal(gpu, 1, hk, 300, d, seed=1), normal(gpu, 1, hk, 300, d, seed=2)
    q, k, v = (normal(gpu, 1, h, d, seed=3 + h) for h in (hq, hk, hk))
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    far_from = 3 * lines + 777  # some way round the ring
    window = 290
    ring, small_ring = lines - sinks, 300 - sinks
    for j in list(range(sinks)) + list(range(far_from - window + 1, far_from)):
        a = j if j < sinks else sinks + (j - sinks) % ring
        b = j if j < sinks else sinks + (j - sinks) % small_ring
        ck[4, :, a], cv[4, :, a] = small_k[0, :, b], small_v[0, :, b]
    pos = torch.tensor([far_from], device=gpu)
    for cache, slot, out in (((ck, cv), 4, o), ((small_k, small_v), 0, o2)):
        need = eg.engram_window_attn_step_workspace_bytes(1, hq, hk, d, cache[0].shape[2])
        eg.engram_window_attn_step(q, k, v, *cache, torch.tensor([slot], device=gpu), pos, out, ws(need, gpu), window,
                                   sinks=sinks, scale=0.1)
    torch.cuda.synchronize()
    same("o", o, o2)
    at, small = sinks + (far_from - sinks) % ring, sinks + (far_from - sinks) % small_ring
    same("line", ck[4, :, at], small_k[0, :, small])
    # all of a cache: constant keys weigh all lines alike, so the output is the values' mean
    ck[4], cv[4] = 0.0, 1.0
    cv[4, :, : lines // 2] = 3.0
    k.zero_()
    v.fill_(1.0)
    need = eg.engram_window_attn_step_workspace_bytes(1, hq, hk, d, lines)
    eg.engram_window_attn_step(q, k, v, ck, cv, torch.tensor([4], device=gpu), torch.tensor([lines - 1], device=gpu), o,
                               ws(need, gpu), lines - sinks, sinks=sinks, scale=0.1)
    assert ((o.double() - 2.0).abs() <= 2.0 ** -8 * 2 + 1e-3).all()


def test_pool_of_states(gpu):
    d, pool = 5120, 220000  # 4.5 GB
    state = torch.empty((pool, d), device=gpu)
    slots = torch.tensor([pool - 1, 0, 214748], device=gpu)
    gate, u = normal(gpu, 3, d, seed=1), normal(gpu, 3, d, seed=2)
    own = torch.randn((3, d), device=gpu)
    state[slots] = own
    h, h2 = torch.empty_like(u), torch.empty_like(u)
    eg.engram_gated_scan_step(gate, u, state, slots, h)
    eg.engram_gated_scan_step(gate, u, own, torch.arange(3, device=gpu), h2)
    torch.cuda.synchronize()
    same("h", h, h2)
    same("state", state[slots], own)
