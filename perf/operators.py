"""The operators beside the Engram gate and GateConv, as cases to be timed.

Three operators, each with its forms for training and for serving:

linear    y = act(x W^T + b) + residual, the projections in front of the gate
          (memory rows to keys and value) and around the token mixers, with its
          backward;
qk        per-head RMS norms of queries and keys with the position rotation in
          the same pass, with its backward;
decay     causal linear attention with a fixed decay for each head: the chunked
          form over ragged prompts, its backward, and the recurrent step of
          single tokens over a pool of states.

`run` computes a case in elementary torch operations in 32 bits (rounded once
at the end), or, where `own` is true, through the library.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- the cases


def listed():
    return [
        # one generated token's memory row (d_mem 2560) projected to the four keys and the shared value
        _linear("linear one token", n=1, k=2560, m=25600, dtype="bf16"),
        # a small decode batch through a gated up-projection of odd width, half precision, pre-activation kept
        _linear("linear few tokens", n=13, k=5120, m=1368, dtype="fp16", act="silu", bias=True, save_z=True),
        # a prompt's output projection added onto the residual stream (hidden 5120)
        _linear("linear prompt", n=4000, k=5120, m=5120, dtype="bf16", bias=True, residual=True),
        # a training step's key/value projection at 4096 tokens, with the activation's gradient
        _linear("linear backward", n=4096, k=2560, m=25600, dtype="bf16", act="gelu", bias=True, backward=True),
        # a decode batch at far positions of a long context, 40 query and 8 key heads
        _qk("qk decode", n=16, hq=40, hk=8, d=128, r=128, dtype="bf16", far=1 << 20),
        # a prompt of 8192 tokens, same heads
        _qk("qk prompt", n=8192, hq=40, hk=8, d=128, r=128, dtype="bf16", far=8192),
        # training: 4 x 2048 tokens, as many keys as queries, half of each head rotated in neighbour pairs
        _qk("qk backward", n=8192, hq=40, hk=40, d=128, r=64, dtype="bf16", far=2048, interleaved=True, backward=True),
        # a ragged fp32 batch with a head size that is no power of two
        _qk("qk backward odd", n=1003, hq=12, hk=3, d=80, r=48, dtype="fp32", far=4096, backward=True),
        # one generated token of one sequence: latency
        _decay("decay one token", form="step", b=1, t=1, h=40, dk=128, dv=128),
        # a decode batch of 64 sequences
        _decay("decay decode", form="step", b=64, t=1, h=40, dk=128, dv=128),
        # seven prompts of uneven length, 8192 tokens at most in one, each continuing from a state
        _decay("decay prompts", form="forward", b=7, t=8192, h=40, dk=128, dv=128, state=True),
        # a training step over uneven sequences
        _decay("decay backward", form="backward", b=5, t=3000, h=32, dk=128, dv=128, state=True),
    ]


def _linear(name, n, k, m, dtype, act="none", bias=False, residual=False, save_z=False, backward=False):
    return {"name": name, "op": "linear", "n": n, "k": k, "m": m, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "save_z": save_z, "backward": backward}


def _qk(name, n, hq, hk, d, r, dtype, far, interleaved=False, backward=False):
    return {"name": name, "op": "qk", "n": n, "hq": hq, "hk": hk, "d": d, "r": r, "dtype": dtype, "far": far,
            "interleaved": interleaved, "backward": backward}


def _decay(name, form, b, t, h, dk, dv, state=False):
    return {"name": name, "op": "decay", "form": form, "b": b, "t": t, "h": h, "dk": dk, "dv": dv, "state": state}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear backward", "qk", "qk backward", "step", "forward", "backward"])
    if kind.startswith("linear"):
        back = kind.endswith("backward")
        n = _log_int(rng, 1, 4096)
        k, m = 8 * _log_int(rng, 8, 640), 8 * _log_int(rng, 8, 1600)
        act = rng.choice(["none", "relu", "silu", "gelu"])
        c = _linear("", n, k, m, rng.choice(["bf16", "bf16", "fp16"]), act, rng.random() < 0.5,
                    not back and rng.random() < 0.5, not back and rng.random() < 0.3, back)
    elif kind.startswith("qk"):
        d = 8 * rng.randint(4, 32)
        r = min(d // 16 * 16, 16 * rng.randint(1, d // 16))
        hk = rng.randint(1, 16)
        c = _qk("", _log_int(rng, 1, 8192), hk * rng.randint(1, 5), hk, d, r, rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                _log_int(rng, 64, 1 << 20), rng.random() < 0.5, kind.endswith("backward"))
        c["n"] = max(1, min(c["n"], 8192 * 80 * 128 // ((c["hq"] + c["hk"]) * d * (2 if c["dtype"] == "fp32" else 1))))
    else:
        h, dk, dv = rng.randint(1, 40), 8 * rng.randint(4, 16), 8 * rng.randint(4, 16)
        if kind == "step":
            c = _decay("", "step", _log_int(rng, 1, 64), 1, h, dk, dv)
        elif kind == "forward":
            b = _log_int(rng, 1, 32)
            c = _decay("", "forward", b, _log_int(rng, 1, 32768 // b), h, dk, dv, rng.random() < 0.5)
        else:
            b = _log_int(rng, 1, 16)
            c = _decay("", "backward", b, _log_int(rng, 1, 12000 // b), min(h, 32), dk, dv, rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(case):
    """The sequences' lengths: the longest first, the others spread below it, none of them round."""
    b, t = case["b"], case["t"]
    return [t] + [max(1, (t * (7 * i + 3)) // (9 * b) - i) for i in range(1, b)]


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case.get("dtype", "bf16")]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "linear":
        n, k, m = case["n"], case["k"], case["m"]
        s["x"] = normal(n, k)
        s["w"] = normal(m, k, std=k ** -0.5)
        if case["backward"]:
            s["grad_y"] = normal(n, m)
            s["z"] = normal(n, m) if case["act"] != "none" else None
        else:
            s["bias"] = normal(m, std=0.1, dtype=torch.float32) if case["bias"] else None
            s["residual"] = normal(n, m) if case["residual"] else None
    elif case["op"] == "qk":
        n, hq, hk, d = case["n"], case["hq"], case["hk"], case["d"]
        # queries, keys and values come out of one projection; q and k are columns of its rows
        packed = normal(n, (hq + 2 * hk) * d)
        s["q"] = packed[:, :hq * d].view(n, hq, d)
        s["k"] = packed[:, hq * d:(hq + hk) * d].view(n, hk, d)
        s["wq"], s["wk"] = (normal(d, std=0.1, mean=1.0, dtype=torch.float32) for _ in range(2))
        start = torch.randint(0, case["far"], (1,), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(n, device="cuda")) % case["far"]
        # the plan of the rotation: each pair's turns for one position, as 64-bit fractions of a turn
        s["freqs"] = torch.tensor([int(_inv_freq(i, case["r"]) / (2 * math.pi) * 2.0 ** 64) for i in range(case["r"] // 2)],
                                  dtype=torch.int64).cuda()
        if case["backward"]:
            s["grad_q_out"], s["grad_k_out"] = normal(n, hq, d), normal(n, hk, d)
    else:
        b, h, dk, dv = case["b"], case["h"], case["dk"], case["dv"]
        s["log_decay"] = _log_decay(h).float().cuda()
        s["scale"] = dk ** -0.5
        if case["form"] == "step":
            s["q"], s["k"], s["v"] = normal(b, h, dk), normal(b, h, dk), normal(b, h, dv)
            # a pool with room for a quarter more sequences, the batch's slots in no order
            pool = b + b // 4 + 1
            s["state"] = normal(pool, h, dk, dv, dtype=torch.float32)
            s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:b].contiguous()
            return s
        lens = _lengths(case)
        n = sum(lens)
        s["q"], s["k"], s["v"] = normal(n, h, dk), normal(n, h, dk), normal(n, h, dv)
        s["lens"] = lens
        s["cu_seqlens"] = torch.tensor([0] + lens).cumsum(0).cuda()
        s["state_in"] = normal(b, h, dk, dv, dtype=torch.float32) if case["state"] else None
        if case["form"] == "backward":
            s["grad_o"] = normal(n, h, dv)
            s["grad_state_out"] = normal(b, h, dk, dv, dtype=torch.float32) if case["state"] else None
    return s


def _inv_freq(i, r, theta=10000.0):
    return theta ** (-2.0 * i / r)


def _log_decay(h):
    """Decays from exp(-1/2) to exp(-1/512) a token, as slopes in a geometric row over the heads."""
    return -torch.pow(2.0, -(1.0 + 8.0 * torch.arange(h, dtype=torch.float64) / h))


# ---------------------------------------------------------------- one pass


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


# --- the plain forms: 32 bits, one rounding


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    return torch.ones_like(z)


def _plain_linear(s):
    c, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    if c["backward"]:
        dz = s["grad_y"].float()
        if c["act"] != "none":
            dz = dz * _act_slope(s["z"].float(), c["act"])
        out = {"grad_x": (dz @ w).to(dt), "grad_w": (dz.t() @ x).to(dt)}
        if c["bias"]:
            out["grad_bias"] = dz.sum(0)
        return out
    z = x @ w.t()
    if c["bias"]:
        z = z + s["bias"]
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["residual"].float()
    out = {"y": y.to(dt)}
    if c["save_z"]:
        out["z"] = z.to(dt)
    return out


def _pairs(x, r, interleaved):
    """The two members of each rotated pair, and what is not rotated."""
    if interleaved:
        p = x[..., :r].reshape(*x.shape[:-1], r // 2, 2)
        return p[..., 0], p[..., 1], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _joined(a, b, rest, interleaved):
    rotated = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((rotated, rest), -1)


def _angles(s):
    r = s["case"]["r"]
    inv = torch.pow(10000.0, -2.0 * torch.arange(r // 2, dtype=torch.float64, device="cuda") / r)
    a = s["positions"].double()[:, None, None] * inv
    return torch.cos(a).float(), torch.sin(a).float()


def _plain_qk(s, eps=1e-6):
    c, dt = s["case"], s["q"].dtype
    r, il = c["r"], c["interleaved"]
    cos, sin = _angles(s)

    def forward(x, w):
        x = x.float()
        a, b, rest = _pairs(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w, r, il)
        return _joined(a * cos - b * sin, a * sin + b * cos, rest, il).to(dt)

    def backward(g, x, w):
        x = x.float()
        a, b, rest = _pairs(g.float(), r, il)
        g = _joined(a * cos + b * sin, b * cos - a * sin, rest, il)
        rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
        u = x * rstd
        gw = g * w
        return (rstd * (gw - u * (u * gw).mean(-1, keepdim=True))).to(dt), (g * u).sum((0, 1))

    if not c["backward"]:
        return {"q_out": forward(s["q"], s["wq"]), "k_out": forward(s["k"], s["wk"])}
    gq, gwq = backward(s["grad_q_out"], s["q"], s["wq"])
    gk, gwk = backward(s["grad_k_out"], s["k"], s["wk"])
    return {"grad_q": gq, "grad_k": gk, "grad_wq": gwq, "grad_wk": gwk}


_CHUNK = 64


def _plain_decay_forward(s, q, k, v, s0):
    """o and the final states in 32 bits: sequences padded to whole chunks, the products inside a chunk direct, the
    chunks' states joined by one product with the powers of the decay."""
    ld, scale, cu = s["log_decay"], s["scale"], s["cu_seqlens"]
    b, n, h = len(s["lens"]), q.shape[0], q.shape[1]
    nc = -(-max(s["lens"]) // _CHUNK)
    at = torch.arange(n, device="cuda")
    seq = torch.searchsorted(cu[1:], at, right=True)
    pos = at - cu[seq]

    def padded(x):
        p = torch.zeros((b, nc * _CHUNK, *x.shape[1:]), device="cuda")
        return p.index_put((seq, pos), x).view(b, nc, _CHUNK, h, x.shape[-1]).permute(0, 3, 1, 2, 4)  # b h nc C d

    def powers(steps):  # decay to the power of each number of steps, 0 for a negative number
        return torch.where(steps >= 0, torch.exp(ld.view(-1, *[1] * steps.dim()) * steps.clamp(min=0)), torch.zeros((), device="cuda"))

    qp, kp, vp = padded(q), padded(k), padded(v)
    i, ci = torch.arange(_CHUNK, device="cuda"), torch.arange(nc, device="cuda")
    inside = ((qp @ kp.transpose(-1, -2).contiguous()) * powers(i[:, None] - i[None, :])[:, None]) @ vp
    last = powers(_CHUNK - 1 - i)[:, None, :, None]
    u = ((kp * last).transpose(-1, -2).contiguous() @ vp).flatten(3)  # b h nc dk*dv
    carried = (powers((ci[:, None] - 1 - ci[None, :]) * _CHUNK) @ u).unflatten(-1, (k.shape[-1], v.shape[-1]))
    if s0 is not None:
        carried = carried + powers(ci * _CHUNK)[..., None, None] * s0[:, :, None]
    o = scale * (inside + powers(i + 1)[:, None, :, None] * (qp @ carried))
    o = o.permute(0, 2, 3, 1, 4).reshape(b, nc * _CHUNK, h, v.shape[-1])[seq, pos]
    left = (cu[1:] - cu[:-1])[seq] - 1 - pos
    final = (padded(k * powers(left).t()[..., None]).flatten(2, 3).transpose(-1, -2).contiguous() @ vp.flatten(2, 3))
    if s0 is not None:
        final = final + powers(cu[1:] - cu[:-1]).t()[..., None, None] * s0
    return o, final


def _plain_decay(s):
    c = s["case"]
    if c["form"] == "step":
        st = s["state"][s["slots"]] * torch.exp(s["log_decay"])[None, :, None, None]
        st = st + s["k"].float()[..., :, None] * s["v"].float()[..., None, :]
        s["state"][s["slots"]] = st
        o = s["scale"] * (s["q"].float()[..., :, None] * st).sum(-2)
        return {"o": o.to(s["q"].dtype), "state": s["state"]}
    q, k, v = (s[x].float() for x in "qkv")
    s0 = s["state_in"]
    if c["form"] == "forward":
        o, final = _plain_decay_forward(s, q, k, v, s0)
        return {"o": o.to(s["q"].dtype), "state_out": final}
    with torch.enable_grad():
        leaves = [x.detach().requires_grad_() for x in ((q, k, v) if s0 is None else (q, k, v, s0))]
        o, final = _plain_decay_forward(s, *leaves[:3], leaves[3] if s0 is not None else None)
        if s0 is None:
            got = torch.autograd.grad(o, leaves, s["grad_o"].float())
        else:
            got = torch.autograd.grad((o, final), leaves, (s["grad_o"].float(), s["grad_state_out"]))
    out = {name: x.to(s["q"].dtype) for name, x in zip(("grad_q", "grad_k", "grad_v"), got)}
    if s0 is not None:
        out["grad_state_in"] = got[3]
    return out


_plain = {"linear": _plain_linear, "qk": _plain_qk, "decay": _plain_decay}


# --- through the library


def _kept(s, **shapes):
    """Output buffers and workspace that a user's program keeps: made at a state's first pass."""
    if "kept" not in s:
        s["kept"] = {n: torch.empty(shape, dtype=dt, device="cuda") for n, (shape, dt) in shapes.items()}
    return s["kept"]


def _own_linear(s):
    import memory_bound_engram_amd as eg
    c, x, w = s["case"], s["x"], s["w"]
    n, k, m, dt = c["n"], c["k"], c["m"], x.dtype
    if c["backward"]:
        out = s.get("kept") or _kept(
            s, grad_x=((n, k), dt), grad_w=((m, k), dt), **({"grad_bias": ((m,), torch.float32)} if c["bias"] else {}),
            workspace=((eg.engram_linear_bwd_workspace_bytes(n, k, m),), torch.uint8))
        eg.engram_linear_bwd(s["grad_y"], x, w, out["grad_x"], out["grad_w"], out["workspace"], z=s["z"],
                             grad_bias=out.get("grad_bias"), act=c["act"])
    else:
        out = s.get("kept") or _kept(
            s, y=((n, m), dt), **({"z": ((n, m), dt)} if c["save_z"] else {}),
            workspace=((eg.engram_linear_fwd_workspace_bytes(n, k, m),), torch.uint8))
        eg.engram_linear_fwd(x, w, out["y"], out["workspace"], bias=s["bias"], residual=s["residual"], z=out.get("z"),
                             act=c["act"])
    return {k_: v for k_, v in out.items() if k_ != "workspace"}


def _own_qk(s):
    import memory_bound_engram_amd as eg
    c, dt = s["case"], s["q"].dtype
    n, hq, hk, d = c["n"], c["hq"], c["hk"], c["d"]
    args = (s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["freqs"])
    if not c["backward"]:
        out = s.get("kept") or _kept(s, q_out=((n, hq, d), dt), k_out=((n, hk, d), dt))
        eg.engram_qk_norm_rope_fwd(*args, out["q_out"], out["k_out"], eps=1e-6, interleaved=c["interleaved"])
        return out
    out = s.get("kept") or _kept(
        s, grad_q=((n, hq, d), dt), grad_k=((n, hk, d), dt), grad_wq=((d,), torch.float32), grad_wk=((d,), torch.float32),
        workspace=((eg.engram_qk_norm_rope_bwd_workspace_bytes(n, hq, hk, d),), torch.uint8))
    eg.engram_qk_norm_rope_bwd(s["grad_q_out"], s["grad_k_out"], *args, out["grad_q"], out["grad_k"], out["grad_wq"],
                               out["grad_wk"], out["workspace"], eps=1e-6, interleaved=c["interleaved"])
    return {k_: v for k_, v in out.items() if k_ != "workspace"}


def _own_decay(s):
    import memory_bound_engram_amd as eg
    c, dt = s["case"], s["q"].dtype
    b, h, dk, dv = c["b"], c["h"], c["dk"], c["dv"]
    q, k, v, ld = s["q"], s["k"], s["v"], s["log_decay"]
    if c["form"] == "step":
        out = s.get("kept") or _kept(s, o=((b, h, dv), dt))
        eg.engram_decay_attn_step(q, k, v, ld, s["state"], s["slots"], out["o"], scale=s["scale"])
        return {"o": out["o"], "state": s["state"]}
    n = q.shape[0]
    states = ((b, h, dk, dv), torch.float32)
    if c["form"] == "forward":
        out = s.get("kept") or _kept(
            s, o=((n, h, dv), dt), state_out=states,
            workspace=((eg.engram_decay_attn_fwd_workspace_bytes(n, b, h, dk, dv),), torch.uint8))
        eg.engram_decay_attn_fwd(q, k, v, ld, s["cu_seqlens"], out["o"], out["workspace"], scale=s["scale"],
                                 state_in=s["state_in"], state_out=out["state_out"])
    else:
        out = s.get("kept") or _kept(
            s, grad_q=((n, h, dk), dt), grad_k=((n, h, dk), dt), grad_v=((n, h, dv), dt),
            **({"grad_state_in": states} if c["state"] else {}),
            workspace=((eg.engram_decay_attn_bwd_workspace_bytes(n, b, h, dk, dv),), torch.uint8))
        eg.engram_decay_attn_bwd(s["grad_o"], q, k, v, ld, s["cu_seqlens"], out["grad_q"], out["grad_k"], out["grad_v"],
                                 out["workspace"], scale=s["scale"], state_in=s["state_in"],
                                 grad_state_out=s["grad_state_out"], grad_state_in=out.get("grad_state_in"))
    return {k_: v_ for k_, v_ in out.items() if k_ != "workspace"}


_own = {"linear": _own_linear, "qk": _own_qk, "decay": _own_decay}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "linear":
        n, k, m, e = case["n"], case["k"], case["m"], _SIZE[case["dtype"]]
        rows = n * k * e + m * k * e
        if case["backward"]:
            return {"bytes": 2 * rows + n * m * e * (2 if case["act"] != "none" else 1) + (4 * m if case["bias"] else 0),
                    "flops": 4 * n * k * m}
        return {"bytes": rows + n * m * e * (1 + case["residual"] + case["save_z"]) + (4 * m if case["bias"] else 0),
                "flops": 2 * n * k * m}
    if case["op"] == "qk":
        values = case["n"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": values * _SIZE[case["dtype"]] * (3 if case["backward"] else 2) + 8 * case["n"] + 8 * case["d"],
                "flops": values * (20 if case["backward"] else 10)}
    h, dk, dv, b = case["h"], case["dk"], case["dv"], case["b"]
    if case["form"] == "step":
        return {"bytes": b * h * (2 * 4 * dk * dv + 2 * (2 * dk + 2 * dv)), "flops": 5 * b * h * dk * dv}
    n = sum(_lengths(case))
    states = b * h * dk * dv * 4
    if case["form"] == "forward":
        return {"bytes": n * h * 2 * (2 * dk + 2 * dv) + states * (2 if case["state"] else 1), "flops": 4 * n * h * dk * dv}
    return {"bytes": n * h * 2 * (4 * dk + 3 * dv) + (states * 3 if case["state"] else 0), "flops": 10 * n * h * dk * dv}


# ---------------------------------------------------------------- 64 bits, from the definitions


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return _exact[case["op"]](case, s)


def _exact_linear(c, s):
    x, w = s["x"].double(), s["w"].double()
    act = c["act"]
    if c["backward"]:
        g = s["grad_y"].double()
        if act != "none":
            z = s["z"].double()
            if act == "relu":
                g = torch.where(z > 0, g, torch.zeros_like(g))
            elif act == "silu":
                p = torch.sigmoid(z)
                g = g * (p + z * p * torch.sigmoid(-z))
            else:
                g = g * (0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi))
        out = {"grad_x": torch.mm(g, w), "grad_w": torch.mm(g.t(), x)}
        if c["bias"]:
            out["grad_bias"] = torch.mv(g.t(), torch.ones(c["n"], dtype=torch.float64, device="cuda"))
        return out
    z = torch.mm(x, w.t())
    if c["bias"]:
        z += s["bias"].double()
    y = {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
         "gelu": lambda: z * 0.5 * torch.erfc(-z / math.sqrt(2.0))}[act]()
    if c["residual"]:
        y = y + s["residual"].double()
    return {"y": y, "z": z} if c["save_z"] else {"y": y}


def _exact_qk(c, s, eps=1e-6):
    d, r = c["d"], c["r"]
    # the rotation as a complex factor of each pair; the rest of the head turns by nothing
    turn = torch.tensor([_inv_freq(i, r) for i in range(r // 2)], dtype=torch.float64, device="cuda")
    ang = s["positions"].double()[:, None] * turn
    factor = torch.polar(torch.ones_like(ang), ang)[:, None, :]
    idx = torch.arange(r, device="cuda").view(-1, 2) if c["interleaved"] else torch.arange(r, device="cuda").view(2, -1).t()

    def rotate(y, f):
        y = y.clone()
        p = torch.complex(y[..., idx[:, 0]], y[..., idx[:, 1]]) * f
        y[..., idx[:, 0]], y[..., idx[:, 1]] = p.real, p.imag
        return y

    def norm(x):
        return (x.square().sum(-1, keepdim=True) / d + eps) ** -0.5

    if not c["backward"]:
        return {o: rotate(s[x].double() * norm(s[x].double()) * s[w].double(), factor)
                for o, x, w in (("q_out", "q", "wq"), ("k_out", "k", "wk"))}
    out = {}
    for x_, w_, g_ in (("q", "wq", "grad_q_out"), ("k", "wk", "grad_k_out")):
        x, w = s[x_].double(), s[w_].double()
        g = rotate(s[g_].double(), factor.conj())
        inv = norm(x)
        gw = g * w
        out["grad_" + x_] = inv * gw - x * inv ** 3 * (x * gw).sum(-1, keepdim=True) / d
        out["grad_" + w_] = (g * x * inv).flatten(0, 1).sum(0)
    return out


def _exact_decay(c, s):
    """The recurrence itself, token after token, all sequences side by side."""
    lam = torch.exp(_log_decay(c["h"]).float().double()).cuda()[None, :, None, None]
    scale = s["scale"]
    q, k, v = (s[x].double() for x in "qkv")
    if c["form"] == "step":
        state = s["state"].double()
        st = lam * state[s["slots"]] + torch.einsum("bhk,bhv->bhkv", k, v)
        state[s["slots"]] = st
        return {"o": scale * torch.einsum("bhk,bhkv->bhv", q, st), "state": state}
    lens, cu = s["lens"], s["cu_seqlens"]
    if max(lens) * len(lens) * c["h"] * c["dk"] * c["dv"] > 6e10 or max(lens) > 40000:
        return None
    b, h, dk, dv = c["b"], c["h"], c["dk"], c["dv"]
    st = torch.zeros((b, h, dk, dv), dtype=torch.float64, device="cuda") if s["state_in"] is None else s["state_in"].double()
    o = torch.empty((q.shape[0], h, dv), dtype=torch.float64, device="cuda")
    back = c["form"] == "backward"
    if back:
        do = s["grad_o"].double()
        dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    order = sorted(range(b), key=lambda i: -lens[i])  # the sequences still running are a prefix of this order
    first = cu[:-1][torch.tensor(order, device="cuda")]
    st = st[torch.tensor(order, device="cuda")].contiguous()
    alive = [sum(n > t for n in lens) for t in range(max(lens))]
    for t, a in enumerate(alive):
        i = first[:a] + t
        x = st[:a]
        x.mul_(lam).add_(k[i][..., :, None] * v[i][..., None, :])
        if back:
            dq[i] = scale * (x * do[i][..., None, :]).sum(-1)
        else:
            o[i] = scale * (q[i][..., :, None] * x).sum(-2)
    inverse = torch.empty(b, dtype=torch.int64, device="cuda")
    inverse[torch.tensor(order, device="cuda")] = torch.arange(b, device="cuda")
    if not back:
        return {"o": o, "state_out": st[inverse]}
    ds = torch.zeros_like(st) if s["grad_state_out"] is None else s["grad_state_out"].double()[torch.tensor(order, device="cuda")]
    for t in reversed(range(len(alive))):
        a = alive[t]
        i = first[:a] + t
        x = ds[:a]  # the gradient that reaches the state after token t
        x.add_(scale * q[i][..., :, None] * do[i][..., None, :])
        dk_[i] = (x * v[i][..., None, :]).sum(-1)
        dv_[i] = (x * k[i][..., :, None]).sum(-2)
        x.mul_(lam)
    out = {"grad_q": dq, "grad_k": dk_, "grad_v": dv_}
    if c["state"]:
        out["grad_state_in"] = ds[inverse]
    return out


_exact = {"linear": _exact_linear, "qk": _exact_qk, "decay": _exact_decay}
