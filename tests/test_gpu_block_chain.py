"""A hybrid block's layers in a row, as a model uses them: layer norm, packed
projection, query/key norms and rotation, window attention, output projection
with the residual; layer norm, projection to gate and candidate, gated scan,
output projection with the residual; all backwards with the residual stream's
gradient; and serving: prompts, caches and states, then single tokens.

Against the whole formula in 64 bits, under autograd, with no rounding inside.
Each result passes some roundings to bf16, each of which moves a tensor by at
most half a step, 2^-8, of its norm; the layers between pass a random error on
in the proportion in which they pass the tensor, but for the gate: its
rounding moves the state by up to |gate| (h - u) f, here up to four times what
the state's own would.  So n roundings move a result by at most n 2^-8 of its norm:
  forward: normed x (1), q, k, v (3), normed q and k (2), weights (1), o (1), the
  residual stream (1), its norm (1), gate (4), u (1), h (1) and the result (1)
  backward: those, as many gradients, and the rounded weights and their
  gradients of the attention (2)
Every stage by itself is held to bounds of its own elsewhere; here a wrong
column, row, sequence or order shows, as it moves a result by its whole norm."""
from __future__ import annotations

import math

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import poisoned

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -8
FORWARD, BACKWARD = 17, 36
E, HQ, HK, D, C, EPS, THETA = 192, 6, 2, 64, 256, 1e-5, 10000.0
QKV = (HQ + 2 * HK) * D
WINDOW, SINKS = 40, 3


def close(name, got, want, roundings):
    off = (got.double().cpu() - want).norm().item()
    assert off <= U * roundings * want.norm().item(), f"{name}: off by {off:.4g} of {want.norm().item():.4g}"


def heads(packed):
    at, out = 0, []
    for h in (HQ, HK, HK):
        out.append(packed[:, at * D:(at + h) * D].unflatten(1, (h, D)))
        at += h
    return out


class Net:
    def __init__(self, lens, dev, seed=3):
        g = torch.Generator(device=dev).manual_seed(seed)

        def r(*s):
            return torch.randn(s, generator=g, device=dev)
        self.lens, self.n, self.dev = lens, sum(lens), dev
        self.x, self.gy = r(self.n, E).to(BF), r(self.n, E).to(BF)
        self.w1, self.b1, self.w2, self.b2 = 1 + 0.2 * r(E), 0.2 * r(E), 1 + 0.2 * r(E), 0.2 * r(E)
        self.wq, self.wk = 1 + 0.2 * r(D), 1 + 0.2 * r(D)
        self.w_in, self.w_out = (r(QKV, E) * E ** -0.5).to(BF), (r(E, HQ * D) * (HQ * D) ** -0.5).to(BF)
        self.w_gu, self.w_h = (r(2 * C, E) * E ** -0.5).to(BF), (r(E, C) * C ** -0.5).to(BF)
        self.positions = torch.cat([torch.arange(n, device=dev) for n in lens])
        self.freqs = eg.engram_rope_freqs(THETA, D).to(dev)
        self.cu = torch.tensor([0] + lens).cumsum(0).to(dev)
        self.scale = D ** -0.5

    def new(self, *s, dt=BF):
        return poisoned(s, dt, self.dev)

    def ws(self, f, *a):
        return poisoned((max(16, f(*a)),), torch.uint8, self.dev)

    def linear(self, x, w, residual=None):
        y = self.new(x.shape[0], w.shape[0])
        eg.engram_linear_fwd(x, w, y, self.ws(eg.engram_linear_fwd_workspace_bytes, x.shape[0], x.shape[1], w.shape[0]),
                             residual=residual)
        return y

    def linear_back(self, gy, x, w, gx=None):
        gx = self.new(*x.shape) if gx is None else gx
        gw = self.new(*w.shape)
        eg.engram_linear_bwd(gy, x, w, gx, gw, self.ws(eg.engram_linear_bwd_workspace_bytes, x.shape[0], x.shape[1], w.shape[0]))
        return gx, gw

    def norm(self, x, w, b):
        y, saved = self.new(*x.shape), self.new(x.shape[0], 2, dt=torch.float32)
        eg.engram_layer_norm_fwd(x, w, y, b=b, saved=saved, eps=EPS)
        return y, saved

    def norm_back(self, gy, x, w, saved, residual):
        gx, gw, gb = self.new(*x.shape), self.new(E, dt=torch.float32), self.new(E, dt=torch.float32)
        eg.engram_layer_norm_bwd(gy, x, w, saved, gx, self.ws(eg.engram_layer_norm_bwd_workspace_bytes, x.shape[0], E),
                                 grad_w=gw, grad_b=gb, grad_residual=residual)
        return gx, gw, gb

    def rotated(self, qkv, positions):
        q, k, _ = heads(qkv)
        qn, kn = self.new(*q.shape), self.new(*k.shape)
        eg.engram_qk_norm_rope_fwd(q, k, self.wq, self.wk, positions, self.freqs, qn, kn)
        return qn, kn

    def forward(self):
        s = {}
        s["n1"], s["m1"] = self.norm(self.x, self.w1, self.b1)
        s["qkv"] = self.linear(s["n1"], self.w_in)
        s["q"], s["k"] = self.rotated(s["qkv"], self.positions)
        s["o"], s["lse"] = self.new(self.n, HQ, D), self.new(self.n, HQ, dt=torch.float32)
        eg.engram_window_attn_fwd(s["q"], s["k"], heads(s["qkv"])[2], self.cu, s["o"], WINDOW, sinks=SINKS, lse=s["lse"],
                                  scale=self.scale)
        s["x2"] = self.linear(s["o"].flatten(1), self.w_out, residual=self.x)
        s["n2"], s["m2"] = self.norm(s["x2"], self.w2, self.b2)
        s["gu"] = self.linear(s["n2"], self.w_gu)
        s["h"], s["state"] = self.new(self.n, C), self.new(len(self.lens), C, dt=torch.float32)
        eg.engram_gated_scan_fwd(s["gu"][:, :C], s["gu"][:, C:], self.cu, s["h"],
                                 self.ws(eg.engram_gated_scan_fwd_workspace_bytes, self.n, len(self.lens), C),
                                 state_out=s["state"])
        s["y"] = self.linear(s["h"], self.w_h, residual=s["x2"])
        return s

    def backward(self, s):
        g, b = {}, len(self.lens)
        gh, g["w_h"] = self.linear_back(self.gy, s["h"], self.w_h)
        ggu = self.new(self.n, 2 * C)
        eg.engram_gated_scan_bwd(gh, s["gu"][:, :C], s["gu"][:, C:], s["h"], self.cu, ggu[:, :C], ggu[:, C:],
                                 self.ws(eg.engram_gated_scan_bwd_workspace_bytes, self.n, b, C))
        gn, g["w_gu"] = self.linear_back(ggu, s["n2"], self.w_gu)
        gx2, g["w2"], g["b2"] = self.norm_back(gn, s["x2"], self.w2, s["m2"], self.gy)
        go, g["w_out"] = self.linear_back(gx2, s["o"].flatten(1), self.w_out)
        gqkv = self.new(self.n, QKV)
        gq, gk, gv = heads(gqkv)
        gqn, gkn = self.new(*gq.shape), self.new(*gk.shape)
        q, k, v = heads(s["qkv"])
        eg.engram_window_attn_bwd(go.unflatten(1, (HQ, D)), s["q"], s["k"], v, s["o"], s["lse"], self.cu, gqn, gkn, gv,
                                  self.ws(eg.engram_window_attn_bwd_workspace_bytes, self.n, b, HQ, HK, D, WINDOW, SINKS),
                                  WINDOW, sinks=SINKS, scale=self.scale)
        g["wq"], g["wk"] = self.new(D, dt=torch.float32), self.new(D, dt=torch.float32)
        eg.engram_qk_norm_rope_bwd(gqn, gkn, q, k, self.wq, self.wk, self.positions, self.freqs, gq, gk, g["wq"], g["wk"],
                                   self.ws(eg.engram_qk_norm_rope_bwd_workspace_bytes, self.n, HQ, HK, D))
        gn, g["w_in"] = self.linear_back(gqkv, s["n1"], self.w_in)
        g["x"], g["w1"], g["b1"] = self.norm_back(gn, self.x, self.w1, s["m1"], gx2)
        return g

    LEAVES = ("x", "w1", "b1", "w2", "b2", "wq", "wk", "w_in", "w_out", "w_gu", "w_h")

    def formula(self, p):
        turns = torch.tensor([[(t * f % 2 ** 64) / 2.0 ** 64 for f in self.freqs.tolist()] for t in self.positions.tolist()],
                             dtype=torch.float64)
        cos, sin = torch.cos(2 * math.pi * turns)[:, None], torch.sin(2 * math.pi * turns)[:, None]

        def norm(x, w, b):
            x = x - x.mean(1, keepdim=True)
            return x * (x.square().mean(1, keepdim=True) + EPS) ** -0.5 * w + b

        def turned(t, w):
            t = t * (t.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * w
            a, b = t[..., :D // 2], t[..., D // 2:]
            return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        q, k, v = heads(norm(p["x"], p["w1"], p["b1"]) @ p["w_in"].t())
        q, k = turned(q, p["wq"]), turned(k, p["wk"])
        o, at = [], 0
        for n in self.lens:
            i = torch.arange(n)
            ago = i[:, None] - i[None]
            seen = (ago >= 0) & ((ago < WINDOW) | (i[None] < SINKS))
            qs, ks, vs = (t[at:at + n].transpose(0, 1) for t in (q, k, v))
            ks, vs = ks.repeat_interleave(HQ // HK, 0), vs.repeat_interleave(HQ // HK, 0)
            z = (self.scale * qs @ ks.transpose(1, 2)).masked_fill(~seen, -math.inf)
            o.append((torch.softmax(z, -1) @ vs).transpose(0, 1))
            at += n
        x2 = torch.cat(o).flatten(1) @ p["w_out"].t() + p["x"]
        gate, u = (norm(x2, p["w2"], p["b2"]) @ p["w_gu"].t()).split(C, 1)
        f, hs, at, last = torch.sigmoid(gate), [], 0, []
        for n in self.lens:
            h = torch.zeros(C, dtype=torch.float64)
            for t in range(at, at + n):
                h = f[t] * h + torch.sigmoid(-gate[t]) * u[t]
                hs.append(h)
            last.append(h)
            at += n
        return torch.stack(hs) @ p["w_h"].t() + x2, torch.stack(last)


@pytest.mark.parametrize("lens", [[70, 0, 1, 129], [1], [300]], ids=str)
def test_forward_and_backward(gpu, lens):
    net = Net(lens, gpu)
    s = net.forward()
    g = net.backward(s)
    p = {n: getattr(net, n).double().cpu().requires_grad_() for n in net.LEAVES}
    y, state = net.formula(p)
    close("y", s["y"], y.detach(), FORWARD)
    close("state", s["state"], state.detach(), FORWARD)
    y.backward(net.gy.double().cpu())
    for n in net.LEAVES:
        if lens == [1] and n in ("wq", "wk"):
            continue  # one token: the softmax does not depend on them, the gradients are roundings of zero
        close("grad_" + n, g[n], p[n].grad, BACKWARD)


def test_graph_of_a_training_step(gpu):
    net = Net([90, 37], gpu)
    want = net.forward()
    want.update({"g_" + n: t for n, t in net.backward(want).items()})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = net.forward()
        kept.update({"g_" + n: t for n, t in net.backward(kept).items()})
    for _ in range(3):
        for t in kept.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(kept[n], t) for n, t in want.items())
        net.forward()


def test_single_tokens_after_prompts(gpu):
    """Prompts of 50 and 9 tokens, then 30 single tokens of each through caches and states, captured and replayed: what the
    forward over all tokens gives."""
    first, more = [50, 9], 30
    net = Net([n + more for n in first], gpu)
    whole = net.forward()
    start = [0, first[0] + more]
    rows = torch.cat([torch.arange(a, a + n) for a, n in zip(start, first)]).to(gpu)
    prompt = Net(first, gpu)
    for n in net.LEAVES:
        setattr(prompt, n, getattr(net, n))
    prompt.x = net.x[rows].contiguous()
    s = prompt.forward()
    # the same sums in another order or split: a few roundings, each of half a step, apart
    close("prompt", s["y"], whole["y"][rows].double().cpu(), FORWARD)
    capacity = WINDOW + SINKS
    ck, cv = (torch.zeros((3, HK, capacity, D), dtype=BF, device=gpu) for _ in range(2))
    states = torch.zeros((3, C), device=gpu)
    slots = torch.tensor([2, 0], device=gpu)
    eg.engram_window_cache_fill(s["k"], heads(s["qkv"])[2], prompt.cu, slots, ck, cv, sinks=SINKS)
    states[slots] = s["state"]
    x, positions = torch.empty((2, E), dtype=BF, device=gpu), torch.tensor(first, device=gpu)

    def token():
        n1, _ = net.norm(x, net.w1, net.b1)
        qkv = net.linear(n1, net.w_in)
        q, k = net.rotated(qkv, positions)
        o = net.new(2, HQ, D)
        eg.engram_window_attn_step(q, k, heads(qkv)[2], ck, cv, slots, positions, o,
                                   net.ws(eg.engram_window_attn_step_workspace_bytes, 2, HQ, HK, D, capacity), WINDOW,
                                   sinks=SINKS, scale=net.scale)
        x2 = net.linear(o.flatten(1), net.w_out, residual=x)
        n2, _ = net.norm(x2, net.w2, net.b2)
        gu = net.linear(n2, net.w_gu)
        h = net.new(2, C)
        eg.engram_gated_scan_step(gu[:, :C], gu[:, C:], states, slots, h)
        return net.linear(h, net.w_h, residual=x2)
    saved = ck.clone(), cv.clone(), states.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = token()
    for t, was in zip((ck, cv, states), saved):
        t.copy_(was)
    for i in range(more):
        at = torch.tensor([a + n + i for a, n in zip(start, first)], device=gpu)
        x.copy_(net.x[at])
        positions.copy_(torch.tensor([n + i for n in first]))
        graph.replay()
        close(f"token {i}", y, whole["y"][at].double().cpu(), FORWARD)
