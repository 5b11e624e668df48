"""Operators of a hybrid block around the gate, as cases to be timed.

Three operators beside the projections, query/key norms and decay attention of
operators.py, each with its forms for training and for serving:

window    softmax attention over the last `window` tokens and the first `sinks`
          ones of each sequence, shared key heads, over ragged prompts, with its
          backward; and the single-token form over a pool of caches that hold
          just those tokens;
norm      layer norm of each token's row, with its backward (both weight
          gradients, and the residual stream's gradient added);
scan      the gated recurrence h_t = f_t h_{t-1} + (1 - f_t) u_t, f = sigmoid(gate),
          over ragged prompts, with its backward; and its single-token form over
          a pool of states.

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
        # one generated token of one sequence, 40 query and 8 key heads, the cache full: latency
        _window("window one token", form="step", b=1, t=20000, hq=40, hk=8, d=128, window=1024, sinks=4),
        # a decode batch of 64 sequences between 1 and 32768 tokens long
        _window("window decode", form="step", b=64, t=32768, hq=40, hk=8, d=128, window=1024, sinks=4),
        # seven prompts of uneven length, 8192 tokens at most in one
        _window("window prompts", form="forward", b=7, t=8192, hq=40, hk=8, d=128, window=1024, sinks=4),
        # three short prompts in half precision, a head size and a window that are no powers of two, no sinks,
        # the softmax's logarithms kept for a backward
        _window("window prompts odd", form="forward", b=3, t=777, hq=12, hk=3, d=80, window=333, sinks=0, dtype="fp16",
                lse=True),
        # a training step over uneven sequences
        _window("window backward", form="backward", b=5, t=4096, hq=32, hk=8, d=128, window=1024, sinks=4),
        # the norm of a decode batch of 16 tokens at hidden 5120: latency
        _norm("norm decode", n=16, d=5120, dtype="bf16"),
        # a prompt of 8192 tokens
        _norm("norm prompt", n=8192, d=5120, dtype="bf16", bias=True),
        # a training step at 8192 tokens, the residual stream's gradient added
        _norm("norm backward", n=8192, d=5120, dtype="bf16", bias=True, residual=True, backward=True),
        # a ragged fp32 batch of an odd width
        _norm("norm backward odd", n=1003, d=1368, dtype="fp32", backward=True),
        # a decode batch of 64 sequences, 5120 channels: latency
        _scan("scan decode", form="step", b=64, t=1, d=5120),
        # seven prompts of uneven length, 8192 tokens at most in one, each continuing from a state
        _scan("scan prompts", form="forward", b=7, t=8192, d=5120, state=True),
        # a training step over uneven sequences
        _scan("scan backward", form="backward", b=5, t=3000, d=5120, state=True),
    ]


def _window(name, form, b, t, hq, hk, d, window, sinks, dtype="bf16", lse=False):
    return {"name": name, "op": "window", "form": form, "b": b, "t": t, "hq": hq, "hk": hk, "d": d, "window": window,
            "sinks": sinks, "dtype": dtype, "lse": lse}


def _norm(name, n, d, dtype, bias=False, residual=False, backward=False):
    return {"name": name, "op": "norm", "n": n, "d": d, "dtype": dtype, "bias": bias, "residual": residual,
            "backward": backward}


def _scan(name, form, b, t, d, state=False, dtype="bf16"):
    return {"name": name, "op": "scan", "form": form, "b": b, "t": t, "d": d, "state": state, "dtype": dtype}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["window step", "window forward", "window forward", "window backward", "window backward", "norm",
                       "norm backward", "scan step", "scan forward", "scan backward"])
    op, _, form = kind.partition(" ")
    if op == "window":
        hk = rng.randint(1, 8)
        hq, d = hk * rng.randint(1, 5), 8 * rng.randint(4, 16)
        window, sinks = _log_int(rng, 16, 1024), rng.choice([0, 0, rng.randint(1, 64)])
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        if form == "step":
            c = _window("", form, _log_int(rng, 1, 64), _log_int(rng, 1, 1 << 20), hq, hk, d, window, sinks, dtype)
        elif form == "forward":
            b = _log_int(rng, 1, 32)
            c = _window("", form, b, _log_int(rng, 1, 24000 // b), hq, hk, d, window, sinks, dtype, rng.random() < 0.5)
        else:
            b = _log_int(rng, 1, 16)
            c = _window("", form, b, _log_int(rng, 1, 10000 // b), min(hq, 4 * hk), hk, d, window, sinks, dtype)
    elif op == "norm":
        back = bool(form)
        c = _norm("", _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 1024), rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                  rng.random() < 0.5, back and rng.random() < 0.5, back)
        c["n"] = max(1, min(c["n"], 8192 * 5120 // (c["d"] * (2 if c["dtype"] == "fp32" else 1))))
    else:
        d, dtype = 8 * _log_int(rng, 8, 640), rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if form == "step":
            c = _scan("", form, _log_int(rng, 1, 64), 1, d, dtype=dtype)
        else:
            b = _log_int(rng, 1, 32)
            most = (24000 if form == "forward" else 8000) // (2 if dtype == "fp32" else 1) // b
            c = _scan("", form, b, _log_int(rng, 1, most), d, rng.random() < 0.5, dtype)
    del c["name"]
    return c


def _lengths(case):
    """The sequences' lengths: the longest first, the others spread below it, none of them round."""
    b, t = case["b"], case["t"]
    return [t] + [max(1, (t * (7 * i + 3)) // (9 * b) - i) for i in range(1, b)]


def _positions(case):
    """The place of each decode row's token in its sequence: behind that many others."""
    return [n - 1 for n in _lengths(case)]


def _seen(p, window, sinks):
    """How many tokens the one behind p others sees, itself among them."""
    return min(p + 1, window) + min(sinks, max(0, p + 1 - window))


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "window":
        hq, hk, d, b = case["hq"], case["hk"], case["d"], case["b"]
        s["scale"] = d ** -0.5
        if case["form"] == "step":
            n = b
        else:
            s["lens"] = _lengths(case)
            s["cu_seqlens"] = torch.tensor([0] + s["lens"]).cumsum(0).cuda()
            n = sum(s["lens"])
        # queries and keys behind their norms (the queries' weights make the softmax peaked), values as
        # columns of the packed projection
        s["q"], s["k"] = normal(n, hq, d, std=2.0), normal(n, hk, d)
        s["v"] = normal(n, (hq + 2 * hk) * d)[:, (hq + hk) * d:].view(n, hk, d)
        if case["form"] == "step":
            # a pool with room for a quarter more sequences, the batch's slots in no order; a token at place p is in
            # line p of its cache if p < sinks, else in line sinks + (p - sinks) % window
            pool, lines = b + b // 4 + 1, case["window"] + case["sinks"]
            s["cache_k"], s["cache_v"] = normal(pool, hk, lines, d), normal(pool, hk, lines, d)
            s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:b].contiguous()
            s["positions"] = torch.tensor(_positions(case)).cuda()
        if case["form"] == "backward":
            s["o"], s["lse"] = _window_forward(s)
            s["grad_o"] = normal(n, hq, d)
    elif case["op"] == "norm":
        n, d = case["n"], case["d"]
        # a residual stream: tokens of different mean and size, a few channels far larger than the rest
        x = torch.randn((n, d), generator=g, device="cuda")
        x[:, ::397] *= 20.0
        x = x * (0.5 + 3 * torch.rand((n, 1), generator=g, device="cuda"))
        s["x"] = (x + 0.3 * torch.randn((n, 1), generator=g, device="cuda")).to(dt)
        s["w"] = normal(d, std=0.1, mean=1.0, dtype=torch.float32)
        s["b"] = normal(d, std=0.1, dtype=torch.float32) if case["bias"] else None
        if case["backward"]:
            s["grad_y"] = normal(n, d)
            s["grad_residual"] = normal(n, d) if case["residual"] else None
            s["saved"] = _moments(s["x"]).float().contiguous()
    else:
        b, d = case["b"], case["d"]
        if case["form"] == "step":
            pool = b + b // 4 + 1
            s["state"] = normal(pool, d, dtype=torch.float32)
            s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:b].contiguous()
            n = b
        else:
            s["lens"] = _lengths(case)
            s["cu_seqlens"] = torch.tensor([0] + s["lens"]).cumsum(0).cuda()
            n = sum(s["lens"])
            s["state_in"] = normal(b, d, dtype=torch.float32) if case["state"] else None
        # gate and candidate out of one projection; the gate's bias spreads the channels' memories from one to
        # a thousand tokens
        packed = normal(n, 2 * d, std=1.5, dtype=torch.float32)
        packed[:, :d] += 7.0 * torch.arange(d, device="cuda") / d
        packed = packed.to(dt)
        s["gate"], s["u"] = packed[:, :d], packed[:, d:]
        if case["form"] == "backward":
            s["h"] = _scan_forward(s)[0].to(dt)
            s["grad_h"] = normal(n, d)
            s["grad_state_out"] = normal(b, d, dtype=torch.float32) if case["state"] else None
    return s


_EPS = 1e-5


def _moments(x):
    """Mean and inverse deviation of each row, [N, 2]."""
    x = x.double()
    mean = x.mean(1)
    return torch.stack((mean, (x.var(1, unbiased=False) + _EPS) ** -0.5), 1)


# ---------------------------------------------------------------- one pass


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


# --- the plain forms: 32 bits, one rounding


_ROWS = 512  # queries at a time


def _blocks(s):
    """Runs of queries of one sequence with the keys any of them sees, and who of them sees whom."""
    c = s["case"]
    at = 0
    for length in s["lens"]:
        for t0 in range(0, length, _ROWS):
            t1 = min(length, t0 + _ROWS)
            first = max(0, t0 - c["window"] + 1)
            keys = torch.arange(first, t1, device="cuda")
            if first > 0 and c["sinks"] > 0:
                keys = torch.cat((torch.arange(min(first, c["sinks"]), device="cuda"), keys))
            t = torch.arange(t0, t1, device="cuda")[:, None]
            visible = (keys <= t) & ((keys > t - c["window"]) | (keys < c["sinks"]))
            yield slice(at + t0, at + t1), at + keys, visible
        at += length


def _heads(x, times=1):
    """[n, h, d] as [h * times, n, d] in 32 bits."""
    return x.float().transpose(0, 1).repeat_interleave(times, 0).contiguous()


def _weights(s, rows, keys, visible):
    """The softmax of a block and its logarithm's offset, [hq, queries, keys] and [hq, queries]."""
    c = s["case"]
    k = _heads(s["k"][keys], c["hq"] // c["hk"])
    z = s["scale"] * (_heads(s["q"][rows]) @ k.transpose(1, 2).contiguous())
    z = torch.where(visible, z, torch.full((), -math.inf, device="cuda"))
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    return p / total, k, (top + torch.log(total))[..., 0]


def _window_forward(s):
    c = s["case"]
    o = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    for rows, keys, visible in _blocks(s):
        p, _, l = _weights(s, rows, keys, visible)
        o[rows] = (p @ _heads(s["v"][keys], c["hq"] // c["hk"])).transpose(0, 1).to(o.dtype)
        lse[rows] = l.t()
    return o, lse


def _plain_window(s):
    c = s["case"]
    hq, hk, d, dt = c["hq"], c["hk"], c["d"], s["q"].dtype
    if c["form"] == "step":
        window, sinks, pos, slots = c["window"], c["sinks"], s["positions"], s["slots"]
        line = torch.where(pos < sinks, pos, sinks + (pos - sinks) % window)
        s["cache_k"][slots, :, line] = s["k"]
        s["cache_v"][slots, :, line] = s["v"]
        # the place of the token in each line of the cache: the last one up to pos that belongs there
        i = torch.arange(sinks + window, device="cuda")
        place = torch.where(i < sinks, i, pos[:, None] - (pos[:, None] - i) % window)
        visible = (place >= 0) & (place <= pos[:, None]) & ((i < sinks) | (place >= sinks))
        k, v = s["cache_k"][slots].float(), s["cache_v"][slots].float()  # b hk lines d
        q = s["q"].float().view(c["b"], hk, hq // hk, d)
        z = s["scale"] * (q @ k.transpose(2, 3).contiguous())
        z = torch.where(visible[:, None, None], z, torch.full((), -math.inf, device="cuda"))
        p = torch.exp(z - z.amax(-1, keepdim=True))
        o = (p @ v) / p.sum(-1, keepdim=True)
        return {"o": o.view(c["b"], hq, d).to(dt), "cache_k": s["cache_k"], "cache_v": s["cache_v"]}
    if c["form"] == "forward":
        o, lse = _window_forward(s)
        return {"o": o, "lse": lse} if c["lse"] else {"o": o}
    times = hq // hk
    grad_q = torch.empty(s["q"].shape, dtype=dt, device="cuda")
    grad_k, grad_v = (torch.zeros(s["k"].shape, device="cuda") for _ in range(2))
    for rows, keys, visible in _blocks(s):
        p, k, _ = _weights(s, rows, keys, visible)
        do = _heads(s["grad_o"][rows])
        dp = do @ _heads(s["v"][keys], times).transpose(1, 2).contiguous()
        ds = s["scale"] * p * (dp - (p * dp).sum(-1, keepdim=True))
        grad_q[rows] = (ds @ k).transpose(0, 1).to(dt)
        for total, a, b in ((grad_k, ds, _heads(s["q"][rows])), (grad_v, p, do)):
            part = (a.transpose(1, 2).contiguous() @ b).view(hk, times, len(keys), d).sum(1)
            total[keys] = total[keys] + part.transpose(0, 1)
    return {"grad_q": grad_q, "grad_k": grad_k.to(dt), "grad_v": grad_v.to(dt)}


def _plain_norm(s):
    c, x, w, dt = s["case"], s["x"].float(), s["w"], s["x"].dtype
    if not c["backward"]:
        x = x - x.mean(1, keepdim=True)
        y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + _EPS) * w
        return {"y": (y if s["b"] is None else y + s["b"]).to(dt)}
    mean, rstd = s["saved"][:, :1], s["saved"][:, 1:]
    xn = (x - mean) * rstd
    gy = s["grad_y"].float()
    g = gy * w
    gx = rstd * (g - g.mean(1, keepdim=True) - xn * (g * xn).mean(1, keepdim=True))
    if c["residual"]:
        gx = gx + s["grad_residual"].float()
    out = {"grad_x": gx.to(dt), "grad_w": (gy * xn).sum(0)}
    if c["bias"]:
        out["grad_b"] = gy.sum(0)
    return out


_CHUNK = 64


def _recurrence(f, x, seq, pos, lens, s0):
    """h_t = f_t h_{t-1} + x_t of every sequence from s0 (zero if None), and the states behind the last tokens' chunks:
    sequences padded to whole chunks, the chunks by doubling, their ends one after the other."""
    d, b, nc = f.shape[1], len(lens), -(-max(lens) // _CHUNK)

    def padded(v, fill):
        p = torch.full((b, nc * _CHUNK, d), fill, device="cuda")
        return p.index_put((seq, pos), v).view(b, nc, _CHUNK, d)

    a, h = padded(f, 1.0), padded(x, 0.0)
    step = 1
    while step < _CHUNK:
        h = torch.cat((h[:, :, :step], h[:, :, step:] + a[:, :, step:] * h[:, :, :-step]), 2)
        a = torch.cat((a[:, :, :step], a[:, :, step:] * a[:, :, :-step]), 2)
        step *= 2
    carry = torch.zeros((b, d), device="cuda") if s0 is None else s0
    before = torch.empty((b, nc, d), device="cuda")
    for i in range(nc):
        before[:, i] = carry
        carry = a[:, i, -1] * carry + h[:, i, -1]
    h = h + a * before[:, :, None]
    return h.view(b, nc * _CHUNK, d)[seq, pos], carry


def _tokens(s):
    cu = s["cu_seqlens"]
    at = torch.arange(s["gate"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:], at, right=True)
    return cu, at, seq, at - cu[seq]


def _gates(gate):
    """sigmoid(gate) and sigmoid(-gate)."""
    gate = gate.float()
    return 1 / (1 + torch.exp(-gate)), 1 / (1 + torch.exp(gate))


def _scan_forward(s):
    _, _, seq, pos = _tokens(s)
    f, new = _gates(s["gate"])
    # behind a sequence's end the padding has f = 1 and x = 0, so the carried state stays
    return _recurrence(f, new * s["u"].float(), seq, pos, s["lens"], s["state_in"])


def _plain_scan(s):
    c, dt = s["case"], s["gate"].dtype
    if c["form"] == "step":
        f, new = _gates(s["gate"])
        h = f * s["state"][s["slots"]] + new * s["u"].float()
        s["state"][s["slots"]] = h
        return {"h": h.to(dt), "state": s["state"]}
    if c["form"] == "forward":
        h, last = _scan_forward(s)
        return {"h": h.to(dt), "state_out": last}
    cu, at, seq, pos = _tokens(s)
    f, new = _gates(s["gate"])
    b = len(s["lens"])
    s0 = torch.zeros((b, c["d"]), device="cuda") if s["state_in"] is None else s["state_in"]
    first, last = cu[:-1], cu[1:] - 1
    # against time: the factor of a token's gradient is the next token's f, and 1 for what comes from behind the last
    later = torch.ones_like(f)
    later[:-1] = f[1:]
    later[last] = 1.0
    dh, _ = _recurrence(later, s["grad_h"].float(), seq, cu[seq + 1] - 1 - at, s["lens"], s["grad_state_out"])
    before = torch.empty_like(f)
    before[1:] = s["h"][:-1].float()
    before[first] = s0
    out = {"grad_gate": (dh * (before - s["u"].float()) * f * new).to(dt), "grad_u": (dh * new).to(dt)}
    if c["state"]:
        out["grad_state_in"] = (f * dh)[first]
    return out


_plain = {"window": _plain_window, "norm": _plain_norm, "scan": _plain_scan}


# --- through the library


def _kept(s, **shapes):
    """Output buffers and workspace that a user's program keeps: made at a state's first pass."""
    if "kept" not in s:
        s["kept"] = {n: torch.empty(shape, dtype=dt, device="cuda") for n, (shape, dt) in shapes.items()}
    return s["kept"]


def _results(kept):
    return {n: t for n, t in kept.items() if n != "workspace"}


def _own_window(s):
    import memory_bound_engram_amd as eg
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    b, hq, hk, d, window, sinks = (c[x] for x in ("b", "hq", "hk", "d", "window", "sinks"))
    n, dt = q.shape[0], q.dtype
    if c["form"] == "step":
        kept = s.get("kept") or _kept(
            s, o=((b, hq, d), dt),
            workspace=((eg.engram_window_attn_step_workspace_bytes(b, hq, hk, d, window + sinks),), torch.uint8))
        eg.engram_window_attn_step(q, k, v, s["cache_k"], s["cache_v"], s["slots"], s["positions"], kept["o"],
                                   kept["workspace"], window, sinks=sinks, scale=s["scale"])
        return {"o": kept["o"], "cache_k": s["cache_k"], "cache_v": s["cache_v"]}
    if c["form"] == "forward":
        kept = s.get("kept") or _kept(s, o=((n, hq, d), dt), **({"lse": ((n, hq), torch.float32)} if c["lse"] else {}))
        eg.engram_window_attn_fwd(q, k, v, s["cu_seqlens"], kept["o"], window, sinks=sinks, lse=kept.get("lse"),
                                  scale=s["scale"])
        return kept
    kept = s.get("kept") or _kept(
        s, grad_q=((n, hq, d), dt), grad_k=((n, hk, d), dt), grad_v=((n, hk, d), dt),
        workspace=((eg.engram_window_attn_bwd_workspace_bytes(n, b, hq, hk, d, window, sinks),), torch.uint8))
    eg.engram_window_attn_bwd(s["grad_o"], q, k, v, s["o"], s["lse"], s["cu_seqlens"], kept["grad_q"], kept["grad_k"],
                              kept["grad_v"], kept["workspace"], window, sinks=sinks, scale=s["scale"])
    return _results(kept)


def _own_norm(s):
    import memory_bound_engram_amd as eg
    c, x = s["case"], s["x"]
    n, d, dt = c["n"], c["d"], x.dtype
    if not c["backward"]:
        kept = s.get("kept") or _kept(s, y=((n, d), dt))
        eg.engram_layer_norm_fwd(x, s["w"], kept["y"], b=s["b"], eps=_EPS)
        return kept
    kept = s.get("kept") or _kept(
        s, grad_x=((n, d), dt), grad_w=((d,), torch.float32), **({"grad_b": ((d,), torch.float32)} if c["bias"] else {}),
        workspace=((eg.engram_layer_norm_bwd_workspace_bytes(n, d),), torch.uint8))
    eg.engram_layer_norm_bwd(s["grad_y"], x, s["w"], s["saved"], kept["grad_x"], kept["workspace"], grad_w=kept["grad_w"],
                             grad_b=kept.get("grad_b"), grad_residual=s["grad_residual"])
    return _results(kept)


def _own_scan(s):
    import memory_bound_engram_amd as eg
    c, gate, u = s["case"], s["gate"], s["u"]
    b, d, dt, n = c["b"], c["d"], gate.dtype, gate.shape[0]
    if c["form"] == "step":
        kept = s.get("kept") or _kept(s, h=((b, d), dt))
        eg.engram_gated_scan_step(gate, u, s["state"], s["slots"], kept["h"])
        return {"h": kept["h"], "state": s["state"]}
    states = ((b, d), torch.float32)
    if c["form"] == "forward":
        kept = s.get("kept") or _kept(
            s, h=((n, d), dt), state_out=states,
            workspace=((eg.engram_gated_scan_fwd_workspace_bytes(n, b, d),), torch.uint8))
        eg.engram_gated_scan_fwd(gate, u, s["cu_seqlens"], kept["h"], kept["workspace"], state_in=s["state_in"],
                                 state_out=kept["state_out"])
    else:
        kept = s.get("kept") or _kept(
            s, grad_gate=((n, d), dt), grad_u=((n, d), dt), **({"grad_state_in": states} if c["state"] else {}),
            workspace=((eg.engram_gated_scan_bwd_workspace_bytes(n, b, d),), torch.uint8))
        eg.engram_gated_scan_bwd(s["grad_h"], gate, u, s["h"], s["cu_seqlens"], kept["grad_gate"], kept["grad_u"],
                                 kept["workspace"], state_in=s["state_in"], grad_state_out=s["grad_state_out"],
                                 grad_state_in=kept.get("grad_state_in"))
    return _results(kept)


_own = {"window": _own_window, "norm": _own_norm, "scan": _own_scan}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    e = _SIZE[case["dtype"]]
    if case["op"] == "window":
        hq, hk, d, w, sinks = (case[x] for x in ("hq", "hk", "d", "window", "sinks"))
        if case["form"] == "step":
            seen = [_seen(p, w, sinks) for p in _positions(case)]
            # the tokens seen, read; the new one's key and value written; q in and o out
            return {"bytes": e * d * (2 * hk * sum(seen) + case["b"] * (2 * hk + 2 * hq)), "flops": 4 * hq * d * sum(seen)}
        lens = _lengths(case)
        n, pairs = sum(lens), sum(_seen_up_to(length, w, sinks) for length in lens)
        if case["form"] == "forward":
            return {"bytes": n * d * e * (2 * hq + 2 * hk) + (4 * n * hq if case["lse"] else 0), "flops": 4 * pairs * hq * d}
        return {"bytes": n * d * e * (4 * hq + 4 * hk) + 4 * n * hq, "flops": 10 * pairs * hq * d}
    if case["op"] == "norm":
        values, d = case["n"] * case["d"], case["d"]
        weights = 4 * d * (2 if case["bias"] else 1)
        if case["backward"]:
            return {"bytes": values * e * (4 if case["residual"] else 3) + 8 * case["n"] + 4 * d + weights,
                    "flops": 15 * values}
        return {"bytes": values * e * 2 + weights, "flops": 8 * values}
    d, b = case["d"], case["b"]
    if case["form"] == "step":
        return {"bytes": b * d * (3 * e + 8), "flops": 10 * b * d}
    values = sum(_lengths(case)) * d
    if case["form"] == "forward":
        return {"bytes": values * e * 3 + b * d * 4 * (2 if case["state"] else 1), "flops": 10 * values}
    return {"bytes": values * e * 6 + (b * d * 4 * 3 if case["state"] else 0), "flops": 15 * values}


def _seen_up_to(length, window, sinks):
    """The sum of _seen over the places of a sequence."""
    short = min(length, window)
    total = short * (short + 1) // 2 + (length - short) * window
    past = max(0, length - window)  # tokens with something behind their window: 1, 2, ... of them
    few = min(past, sinks)
    return total + few * (few + 1) // 2 + (past - few) * sinks


# ---------------------------------------------------------------- 64 bits, from the definitions


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return _exact[case["op"]](case, s)


def _exact_window(c, s):
    """Every sequence and query head by itself, over the whole square of its tokens."""
    window, sinks, scale, per = c["window"], c["sinks"], s["scale"], c["hq"] // c["hk"]
    q, k, v = (s[x].double() for x in "qkv")
    if c["form"] == "step":
        ck, cv = s["cache_k"].double(), s["cache_v"].double()
        o = torch.empty_like(q)
        for r, (slot, p) in enumerate(zip(s["slots"].tolist(), s["positions"].tolist())):
            def line(j):
                return j if j < sinks else sinks + (j - sinks) % window
            ck[slot, :, line(p)], cv[slot, :, line(p)] = k[r], v[r]
            seen = sorted(set(range(min(sinks, p + 1))) | set(range(max(0, p - window + 1), p + 1)))
            at = torch.tensor([line(j) for j in seen], device="cuda")
            for h in range(c["hk"]):
                heads = slice(h * per, (h + 1) * per)
                w = torch.softmax(scale * torch.mm(q[r, heads], ck[slot, h, at].t()), 1)
                o[r, heads] = torch.mm(w, cv[slot, h, at])
        return {"o": o, "cache_k": ck, "cache_v": cv}
    back = c["form"] == "backward"
    if sum(n * n for n in s["lens"]) * c["hq"] * c["d"] * (10 if back else 4) > 2e14 or max(s["lens"]) > 24000:
        return None
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    gk, gv = torch.zeros_like(k), torch.zeros_like(v)
    do = s["grad_o"].double() if back else None
    at = 0
    for n in s["lens"]:
        i = torch.arange(n, device="cuda")
        ago = i[:, None] - i[None, :]
        hidden = ~((ago >= 0) & ((ago < window) | (i[None, :] < sinks)))
        rows = slice(at, at + n)
        for h in range(c["hq"]):
            kh, vh = k[rows, h // per], v[rows, h // per]
            z = (torch.mm(q[rows, h], kh.t()) * scale).masked_fill_(hidden, -math.inf)
            lse[rows, h] = torch.logsumexp(z, 1)
            w = torch.softmax(z, 1)
            if not back:
                out[rows, h] = torch.mm(w, vh)
                continue
            g = do[rows, h]
            gv[rows, h // per] += torch.mm(w.t(), g)
            w2 = torch.mm(g, vh.t())
            w2 = w * (w2 - (w * w2).sum(1, keepdim=True)) * scale
            out[rows, h] = torch.mm(w2, kh)
            gk[rows, h // per] += torch.mm(w2.t(), q[rows, h])
        at += n
    if back:
        return {"grad_q": out, "grad_k": gk, "grad_v": gv}
    return {"o": out, "lse": lse} if c["lse"] else {"o": out}


def _exact_norm(c, s):
    x, w, d = s["x"].double(), s["w"].double(), c["d"]
    m = _moments(s["x"])
    u = (x - m[:, :1]) * m[:, 1:]
    if not c["backward"]:
        y = u * w
        return {"y": y if s["b"] is None else y + s["b"].double()}
    gy = s["grad_y"].double()
    g = gy * w
    gx = m[:, 1:] / d * (d * g - g.sum(1, keepdim=True) - u * (g * u).sum(1, keepdim=True))
    if c["residual"]:
        gx += s["grad_residual"].double()
    out = {"grad_x": gx, "grad_w": (gy * u).sum(0)}
    if c["bias"]:
        out["grad_b"] = gy.sum(0)
    return out


def _exact_scan(c, s):
    """The recurrence itself, token after token, all sequences side by side."""
    gate, u = s["gate"].double(), s["u"].double()
    f, new = torch.sigmoid(gate), torch.sigmoid(-gate)
    if c["form"] == "step":
        state = s["state"].double()
        h = f * state[s["slots"]] + new * u
        state[s["slots"]] = h
        return {"h": h, "state": state}
    lens, cu, b, d = s["lens"], s["cu_seqlens"], c["b"], c["d"]
    order = torch.tensor(sorted(range(b), key=lambda i: -lens[i]), device="cuda")
    first = cu[:-1][order]  # the sequences still running are a prefix of this order
    alive = [sum(n > t for n in lens) for t in range(max(lens))]
    st = torch.zeros((b, d), dtype=torch.float64, device="cuda") if s["state_in"] is None else s["state_in"].double()[order]
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(b, device="cuda")
    if c["form"] == "forward":
        x, h = new * u, torch.empty_like(u)
        for t, a in enumerate(alive):
            i = first[:a] + t
            h[i] = st[:a].mul_(f[i]).add_(x[i])
        return {"h": h, "state_out": st[inverse]}
    ds = torch.zeros_like(st) if s["grad_state_out"] is None else s["grad_state_out"].double()[order]
    grad_h, h = s["grad_h"].double(), s["h"].double()
    dh, before = torch.empty_like(grad_h), torch.empty_like(h)
    for t in reversed(range(len(alive))):
        a = alive[t]
        i = first[:a] + t
        x = ds[:a]  # the gradient that reaches the state behind token t
        x.add_(grad_h[i])
        dh[i] = x
        before[i] = h[i - 1] if t else st[:a]
        x.mul_(f[i])
    out = {"grad_gate": dh * (before - u) * f * new, "grad_u": dh * new}
    if c["state"]:
        out["grad_state_in"] = ds[inverse]
    return out


_exact = {"window": _exact_window, "norm": _exact_norm, "scan": _exact_scan}
