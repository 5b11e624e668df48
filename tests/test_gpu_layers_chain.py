"""The layers in a row, as a model uses them: a packed projection, the norms
and the rotation of its query and key columns, the decay attention reading the
value columns where they are, the output projection with the residual; then
all backwards, the gradients of the packed row written into its columns.
Against the whole formula in 64 bits, under autograd, with no rounding inside.

Each result passes some roundings to bf16, each of which moves a tensor by at
most half a step, 2^-8, of its norm (2^-8 / sqrt 3 if the roundings are even).
The layers between pass a random error on in the proportion in which they pass
the tensor (weights, queries and keys are random), so n roundings move a result
by at most n 2^-8 of its norm:
  forward: q, k, v (3), normed q and k (2), scores and states (2), o (1)
  backward: those seven, grad_o (1), the backward's scores and states (2), the
  gradients of normed q and k (1), of q, k and v (1), and of x or the weight (1)
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
FORWARD, BACKWARD = 8, 13
E, H, D, EPS, THETA = 192, 4, 64, 1e-6, 10000.0
HD = H * D


def close(name, got, want, roundings, own=None):
    """In norm; `own` is what the result's last rounding is relative to, if not the result itself."""
    off = (got.double() - want).norm().item()
    bound = U * (roundings * want.norm().item() + (0 if own is None else own.norm().item()))
    assert off <= bound, f"{name}: off by {off:.4g}, bound {bound:.4g}, norm {want.norm().item():.4g}"


class Net:
    def __init__(self, lens, tail, dev, seed=3):
        g = torch.Generator(device=dev).manual_seed(seed)

        def r(*s):
            return torch.randn(s, generator=g, device=dev)
        n = sum(lens) + tail
        self.lens, self.n, self.used, self.dev = lens, n, sum(lens), dev
        self.x = r(n, E).to(BF)
        self.w_in, self.b_in = (r(3 * HD, E) * E ** -0.5).to(BF), 0.2 * r(3 * HD)
        self.w_out = (r(E, HD) * HD ** -0.5).to(BF)
        self.wq, self.wk = 1 + 0.2 * r(D), 1 + 0.2 * r(D)
        self.ld = -torch.pow(2.0, -torch.arange(H, device=dev, dtype=torch.float32) - 2)
        self.s0 = 0.3 * r(len(lens), H, D, D)
        self.positions = torch.cat([torch.arange(l, device=dev) + 100 * i for i, l in enumerate(lens)] +
                                   [torch.zeros(tail, dtype=torch.int64, device=dev)])
        self.freqs = eg.engram_rope_freqs(THETA, D).to(dev)
        self.cu = torch.tensor([0] + lens).cumsum(0).to(dev)
        self.gy, self.gs = r(n, E).to(BF), 0.3 * r(len(lens), H, D, D)
        self.gy[self.used:] = 0
        self.scale = D ** -0.5

    def buffers(self):
        n, dev, b = self.n, self.dev, len(self.lens)

        def ws(need):
            return poisoned((max(need, 16),), torch.uint8, dev)

        def new(*s, dt=BF):
            return poisoned(s, dt, dev)
        o = dict(qkv=new(n, 3 * HD), qk=new(n, 2 * HD), o=new(n, H, D), y=new(n, E), s=new(b, H, D, D, dt=torch.float32),
                 gw_out=new(E, HD), go=new(n, H, D), gqk=new(n, 2 * HD), gqkv=new(n, 3 * HD), gx=new(n, E),
                 gw_in=new(3 * HD, E), gs0=new(b, H, D, D, dt=torch.float32))
        for s, m in (("gb_in", 3 * HD), ("gwq", D), ("gwk", D)):
            o[s] = new(m, dt=torch.float32)
        o["ws"] = [ws(f(*a)) for f, a in ((eg.engram_linear_fwd_workspace_bytes, (n, E, 3 * HD)),
                                          (eg.engram_decay_attn_fwd_workspace_bytes, (n, b, H, D, D)),
                                          (eg.engram_linear_fwd_workspace_bytes, (n, HD, E)),
                                          (eg.engram_linear_bwd_workspace_bytes, (n, HD, E)),
                                          (eg.engram_decay_attn_bwd_workspace_bytes, (n, b, H, D, D)),
                                          (eg.engram_qk_norm_rope_bwd_workspace_bytes, (n, H, H, D)),
                                          (eg.engram_linear_bwd_workspace_bytes, (n, E, 3 * HD)))]
        return o

    def columns(self, packed, parts):
        return [packed[:, i * HD:(i + 1) * HD].unflatten(1, (H, D)) for i in range(parts)]

    def forward(self, o):
        # rows behind the last sequence take part in the products around the mixer, which leaves them alone
        o["o"].zero_()
        eg.engram_linear_fwd(self.x, self.w_in, o["qkv"], workspace=o["ws"][0], bias=self.b_in)
        q, k, v = self.columns(o["qkv"], 3)
        qn, kn = self.columns(o["qk"], 2)
        eg.engram_qk_norm_rope_fwd(q, k, self.wq, self.wk, self.positions, self.freqs, qn, kn, eps=EPS)
        eg.engram_decay_attn_fwd(qn, kn, v, self.ld, self.cu, o["o"], o["ws"][1], scale=self.scale, state_in=self.s0,
                                 state_out=o["s"])
        eg.engram_linear_fwd(o["o"].flatten(1), self.w_out, o["y"], workspace=o["ws"][2], residual=self.x)

    def backward(self, o):
        o["gqk"].zero_()
        o["gqkv"].zero_()
        q, k, v = self.columns(o["qkv"], 3)
        qn, kn = self.columns(o["qk"], 2)
        gq, gk, gv = self.columns(o["gqkv"], 3)
        gqn, gkn = self.columns(o["gqk"], 2)
        eg.engram_linear_bwd(self.gy, o["o"].flatten(1), self.w_out, o["go"].flatten(1), o["gw_out"], o["ws"][3])
        eg.engram_decay_attn_bwd(o["go"], qn, kn, v, self.ld, self.cu, gqn, gkn, gv, o["ws"][4], scale=self.scale,
                                 state_in=self.s0, grad_state_out=self.gs, grad_state_in=o["gs0"])
        eg.engram_qk_norm_rope_bwd(gqn, gkn, q, k, self.wq, self.wk, self.positions, self.freqs, gq, gk, o["gwq"],
                                   o["gwk"], o["ws"][5], eps=EPS)
        eg.engram_linear_bwd(o["gqkv"], self.x, self.w_in, o["gx"], o["gw_in"], o["ws"][6], grad_bias=o["gb_in"])

    def leaves64(self):
        return {s: getattr(self, s).double().cpu().requires_grad_() for s in ("x", "w_in", "b_in", "w_out", "wq", "wk", "s0")}

    def formula(self, p):
        """y and the states behind the sequences, in 64 bits; the attention in its quadratic form."""
        table = self.freqs.tolist()
        turns = torch.tensor([[((t * f) & (2 ** 64 - 1)) / 2.0 ** 64 for f in table] for t in self.positions.tolist()],
                             dtype=torch.float64)
        cos, sin = torch.cos(2 * math.pi * turns)[:, None], torch.sin(2 * math.pi * turns)[:, None]

        def norm_turn(t, w):
            t = t * (t.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
            a, b = t[..., :D // 2], t[..., D // 2:]
            return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        q, k, v = (p["x"] @ p["w_in"].t() + p["b_in"]).unflatten(1, (3, H, D)).unbind(1)
        q, k = norm_turn(q, p["wq"]), norm_turn(k, p["wk"])
        ld = self.ld.double().cpu()
        os, states, at = [], [], 0
        for b, l in enumerate(self.lens):
            qb, kb, vb = (t[at:at + l].transpose(0, 1) for t in (q, k, v))  # [H][l][D]
            t = torch.arange(l, dtype=torch.float64)
            ago = t[:, None] - t[None]
            decay = torch.where(ago >= 0, torch.exp(ld[:, None, None] * ago.clamp(min=0)), torch.zeros(()).double())
            past = torch.exp(ld[:, None, None] * (t + 1)[None, :, None])
            os.append((self.scale * (((qb @ kb.transpose(1, 2)) * decay) @ vb + past * (qb @ p["s0"][b]))).transpose(0, 1))
            left = torch.exp(ld[:, None, None] * (l - 1 - t)[None, :, None])
            states.append(torch.exp(ld * l)[:, None, None] * p["s0"][b] + (kb * left).transpose(1, 2) @ vb)
            at += l
        mixed = torch.cat(os + [torch.zeros((self.n - at, H, D), dtype=torch.float64)]).flatten(1) @ p["w_out"].t()
        return mixed + p["x"], torch.stack(states), mixed


LENS = [([70, 0, 1, 129], 3), ([1], 0), ([513], 0), ([64, 64, 17], 300)]


@pytest.mark.parametrize("lens,tail", LENS)
def test_forward_and_backward(gpu, lens, tail):
    print(f"chain lens={lens} tail={tail}", flush=True)
    net = Net(lens, tail, gpu)
    o = net.buffers()
    net.forward(o)
    net.backward(o)
    torch.cuda.synchronize()
    p = net.leaves64()
    y, s, mixed = net.formula(p)
    ((y * net.gy.double().cpu()).sum() + (s * net.gs.double().cpu()).sum()).backward()
    got = {k: t.cpu() for k, t in o.items() if k != "ws"}
    close("mixer", got["y"].double() - p["x"].detach(), mixed.detach(), FORWARD, own=y.detach())
    close("states", got["s"], s.detach(), FORWARD)
    close("grad_w_out", got["gw_out"], p["w_out"].grad, BACKWARD)
    close("grad_w_in", got["gw_in"], p["w_in"].grad, BACKWARD)
    close("grad_b_in", got["gb_in"], p["b_in"].grad, BACKWARD)
    close("grad_wq", got["gwq"], p["wq"].grad, BACKWARD)
    close("grad_wk", got["gwk"], p["wk"].grad, BACKWARD)
    close("grad_state", got["gs0"], p["s0"].grad, BACKWARD)
    close("grad_x", got["gx"], p["x"].grad - net.gy.double().cpu(), BACKWARD)  # the residual's share is grad_y itself


def test_a_prompt_then_single_tokens(gpu):
    """The prompt's last tokens through the decode forms (few-row products, one
    step of the states) give what the whole sequence gives."""
    lens, last = [40, 97], 3
    net = Net(lens, 0, gpu, seed=5)
    net.s0.zero_()
    y, s, mixed = (t.detach() for t in net.formula(net.leaves64()))
    at = net.cu.tolist()
    short = Net([l - last for l in lens], 0, gpu, seed=5)
    rows = torch.cat([torch.arange(at[b], at[b + 1] - last, device=gpu) for b in range(2)])
    for name in ("w_in", "b_in", "w_out", "wq", "wk", "ld", "s0"):
        setattr(short, name, getattr(net, name))
    short.x, short.positions = net.x[rows].contiguous(), net.positions[rows].contiguous()
    o = short.buffers()
    short.forward(o)
    pool = poisoned((5, H, D, D), torch.float32, gpu)
    slots = torch.tensor([3, 1], device=gpu)
    pool[slots] = o["s"]
    want_rows = [rows]
    got = [o["y"]]
    for t in range(last):
        now = torch.tensor([at[b + 1] - last + t for b in range(2)], device=gpu)
        x = net.x[now].contiguous()
        qkv, qk = poisoned((2, 3 * HD), BF, gpu), poisoned((2, 2 * HD), BF, gpu)
        mix, out = poisoned((2, H, D), BF, gpu), poisoned((2, E), BF, gpu)
        eg.engram_linear_fwd(x, net.w_in, qkv, bias=net.b_in)
        q, k, v = net.columns(qkv, 3)
        qn, kn = net.columns(qk, 2)
        eg.engram_qk_norm_rope_fwd(q, k, net.wq, net.wk, net.positions[now].contiguous(), net.freqs, qn, kn, eps=EPS)
        eg.engram_decay_attn_step(qn, kn, v, net.ld, pool, slots, mix, scale=net.scale)
        eg.engram_linear_fwd(mix.flatten(1), net.w_out, out, residual=x)
        want_rows.append(now)
        got.append(out)
    torch.cuda.synchronize()
    for r, g in zip(want_rows, got):
        r = r.cpu()
        close("mixer", g.cpu().double() - net.x.cpu()[r].double(), mixed[r], FORWARD, own=y[r])
    close("states", pool[slots].cpu(), s, FORWARD)
    assert bool((pool[[0, 2, 4]].view(torch.uint8) == 0xFF).all())


def test_graph(gpu):
    """The whole row, forward and backward, captured and replayed between eager runs on other buffers."""
    net = Net([70, 0, 1, 129], 3, gpu)
    eager, held = net.buffers(), net.buffers()
    net.forward(eager)
    net.backward(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        net.forward(held)
        net.backward(held)
    other = net.buffers()
    for _ in range(3):
        for k, t in held.items():
            if k != "ws":
                t.view(torch.uint8).fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for k, t in held.items():
            if k != "ws":
                assert torch.equal(t.view(torch.uint8), eager[k].view(torch.uint8)), k
        net.forward(other)
        net.backward(other)
        torch.cuda.synchronize()
        for k, t in other.items():
            if k != "ws":
                assert torch.equal(t.view(torch.uint8), eager[k].view(torch.uint8)), k
