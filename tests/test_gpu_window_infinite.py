"""Values that are not finite, in what rows see and beside it at once: a result that the
definition makes of finite values alone is as without them, all others are infinite or
NaN, and the calls take no longer than a few ordinary ones."""
from __future__ import annotations

import math
import time

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import check
from test_gpu_window_attn import backward64, case, forward64, run_backward, run_forward, visible

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def bad(x):
    return ~torch.isfinite(x)


def finite(x):
    return torch.where(bad(x), torch.zeros_like(x), x)


def held(name, got, want, bound, ok):
    """Within the bound where the definition is finite; elsewhere not finite either."""
    assert not torch.isfinite(got[~ok]).any(), name
    check(name, torch.where(ok, got.double(), want), want, bound)


def touched(x, places, value):
    x = x.clone()
    for token, column in places:
        x[token, :, column] = value
    return x


def spans(c):
    at = 0
    for n in c["lens"]:
        if n:
            yield slice(at, at + n)
        at += n


def any_seen(c, of_tokens):
    """Of [N, heads or 1, ...] truth values of tokens, whether a row sees one that is true: [N, ...] for each head."""
    out = torch.zeros_like(of_tokens)
    for rows in spans(c):
        seen = visible(rows.stop - rows.start, c["window"], c["sinks"]).to(of_tokens.device).double()
        x = of_tokens[rows].double()
        out[rows] = (seen @ x.flatten(1)).view(x.shape) > 0
    return out


def any_sees(c, of_rows):
    """Of truth values of rows, whether one that sees a token is true."""
    out = torch.zeros_like(of_rows)
    for rows in spans(c):
        seen = visible(rows.stop - rows.start, c["window"], c["sinks"]).to(of_rows.device).double()
        x = of_rows[rows].double()
        out[rows] = (seen.t() @ x.flatten(1)).view(x.shape) > 0
    return out


# some columns of a few tokens, early, in the middle and late, beside each other and far apart
PLACES = [(10, 3), (11, 7), (150, 3), (290, 1), (291, 4), (299, 1), (390, -1), (532, 0)]


def check_values(c, value, dev):
    """In v."""
    hk, per = c["hk"], c["hq"] // c["hk"]
    (o64, eo), _ = forward64(c)
    c["v"] = touched(c["v"], PLACES, value)
    o, lse = run_forward(c, dev)
    ok = ~any_seen(c, bad(c["v"])).repeat_interleave(per, 1)
    held("o", o, o64, eo, ok)
    # the backward, from what the forward gave
    clean = {**c, "v": finite(c["v"])}
    want = backward64(clean, torch.where(ok, o, torch.zeros_like(o)), lse)
    gq, gk, gv = run_backward(c, o, lse, dev)
    fine = ok.all(2)  # rows that see no such value: their delta is finite
    check("grad_q", gq[fine], want[0][0][fine], 2 * want[0][1][fine])
    assert not torch.isfinite(gq[~fine]).any()
    rows = ~fine.view(-1, hk, per).all(2)
    lost = any_sees(c, rows) | bad(c["v"]).any(2)  # dk of tokens that such a row sees
    check("grad_k", gk[~lost], want[1][0][~lost], 2 * want[1][1][~lost])
    assert not torch.isfinite(gk[lost]).any()
    check("grad_v", gv, want[2][0], 2 * want[2][1])  # weights do not know of v


def check_gradients(c, value, dev):
    """In grad_o."""
    hk, per = c["hk"], c["hq"] // c["hk"]
    o, lse = run_forward(c, dev)
    want = backward64(c, o, lse)
    c["go"] = touched(c["go"], PLACES, value)
    gq, gk, gv = run_backward(c, o, lse, dev)
    rows = bad(c["go"]).any(2)
    check("grad_q", gq[~rows], want[0][0][~rows], 2 * want[0][1][~rows])
    assert not torch.isfinite(gq[rows]).any()
    lost = any_sees(c, rows.view(-1, hk, per).any(2))
    check("grad_k", gk[~lost], want[1][0][~lost], 2 * want[1][1][~lost])
    assert not torch.isfinite(gk[lost]).any()
    ok = ~any_sees(c, bad(c["go"]).view(-1, hk, per, c["d"]).any(2))
    held("grad_v", gv, want[2][0], 2 * want[2][1], ok)


@pytest.mark.parametrize("check_them", [check_values, check_gradients], ids=["values", "gradients"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("window,sinks", [(40, 5), (150, 0), (1 << 40, 0), (3, 100)])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_seen_and_not_seen(gpu, window, sinks, dtype, value, check_them):
    check_them(case([200, 333], 4, 2, 72, dtype, gpu, window, sinks, seed=1), value, gpu)


@pytest.mark.parametrize("check_them", [check_values, check_gradients], ids=["values", "gradients"])
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 8), (3, 3, 128), (5, 1, 64), (32, 1, 40), (7, 7, 120)])
def test_heads(gpu, hq, hk, d, check_them):
    for dtype in (BF, FP):
        print(f"infinite heads {hq}/{hk} d={d} {dtype}", flush=True)
        check_them(case([200, 0, 333], hq, hk, d, dtype, gpu, 60, 9, seed=d, apart=True), math.inf, gpu)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("window,sinks", [(40, 5), (150, 0), (1 << 40, 0)])
def test_keys(gpu, window, sinks, dtype):
    """An infinite key's score is infinite: above, the row is lost; below, its weight is 0, and only that column of
    dq is 0 times infinity."""
    lens, at = [200, 333], (150, 300)
    c = case(lens, 4, 2, 72, dtype, gpu, window, sinks, seed=3)
    o, lse = run_forward(c, gpu)
    (o64, eo), _ = forward64(c)
    want = backward64(c, o, lse)
    c["k"] = touched(c["k"], [(x, 3) for x in at], math.inf)
    o2, lse2 = run_forward(c, gpu)
    gq, gk, gv = run_backward(c, o2, lse2, gpu)
    sees = any_seen(c, bad(c["k"]).any(2))[:, :1]  # [N, 1]
    above = sees & (c["q"][:, :, 3] > 0)
    below = sees & ~above
    assert not torch.isfinite(o2[above]).any() and not torch.isfinite(gq[above]).any()
    check("o", o2[~sees[:, 0]], o64[~sees[:, 0]], eo[~sees[:, 0]])
    check("grad_q", gq[~sees[:, 0]], want[0][0][~sees[:, 0]], 2 * want[0][1][~sees[:, 0]])
    assert torch.isfinite(o2[below]).all() and torch.isfinite(lse2[below]).all()
    column = torch.arange(72, device=gpu) == 3
    assert not torch.isfinite(gq[below][:, column]).any() and torch.isfinite(gq[below][:, ~column]).all()
    lost = any_sees(c, above.view(-1, 2, 2).any(2))  # tokens that a lost row sees
    assert torch.isfinite(gk[~lost]).all() and torch.isfinite(gv[~lost]).all()
    assert not torch.isfinite(gk[lost]).any() and not torch.isfinite(gv[lost]).any()


def test_finite_values_near_the_largest(gpu):
    """Weights that follow the maximum loosely times values near bf16's largest pass fp32's range; the output does not."""
    c = case([200], 2, 1, 64, BF, gpu, 64, 2, std=1.0, seed=3)
    c["v"] = (c["v"].float().abs() * 2.0 ** 123).to(BF)
    (o64, eo), _ = forward64(c)
    o, _ = run_forward(c, gpu)
    check("o", o, o64, eo)


def seconds(call):
    call()
    torch.cuda.synchronize()
    best = math.inf
    for _ in range(3):
        began = time.perf_counter()
        call()
        torch.cuda.synchronize()
        best = min(best, time.perf_counter() - began)
    return best


@pytest.mark.parametrize("lens,window,sinks", [([8192, 700], 1024, 4), ([8000], 1 << 40, 0)], ids=["window", "all of the past"])
def test_one_value_does_not_hold_up_a_call(gpu, lens, window, sinks):
    """Five times the ordinary time and a millisecond: what is not finite by the definition is looked for by reading v
    or grad_o once more for every 32 rows or keys, not computed again row by row."""
    hq, hk, d = 16, 4, 128
    c = case(lens, hq, hk, d, FP, gpu, window, sinks, seed=4)
    n, b = c["n"], len(lens)
    o, lse = torch.empty_like(c["q"]), torch.empty((n, hq), device=gpu)
    grads = [torch.empty_like(c[x]) for x in "qkv"]
    ws = torch.empty(eg.engram_window_attn_bwd_workspace_bytes(n, b, hq, hk, d, window, sinks), dtype=torch.uint8, device=gpu)

    def fwd(c):
        eg.engram_window_attn_fwd(c["q"], c["k"], c["v"], c["cu"], o, window, sinks=sinks, lse=lse, scale=c["scale"])

    def bwd(c):
        eg.engram_window_attn_bwd(c["go"], c["q"], c["k"], c["v"], o, lse, c["cu"], *grads, ws, window, sinks=sinks,
                                  scale=c["scale"])
    base = seconds(lambda: fwd(c)), seconds(lambda: bwd(c))
    took = {}
    for at in (10, 4000, 7990):
        go = touched(c["go"], [(at, 5)], math.inf)
        took["go", at] = seconds(lambda: bwd({**c, "go": go})), base[1]
    for at in (10, 4000, 7990):
        v = touched(c["v"], [(at, 5)], math.inf)
        took["v", at] = seconds(lambda: fwd({**c, "v": v})), base[0]
    # every row (or value) with one column, and one with another
    go, v = touched(c["go"], [(slice(None), 7), (4000, 5)], math.inf), touched(c["v"], [(slice(None), 7), (4000, 5)], math.inf)
    took["go", "all"] = seconds(lambda: bwd({**c, "go": go})), base[1]
    took["v", "all"] = seconds(lambda: fwd({**c, "v": v})), base[0]
    for at, (t, ordinary) in took.items():
        print(f"infinite {at}: {t * 1e3:.2f} ms, ordinary {ordinary * 1e3:.2f} ms", flush=True)
    assert all(t <= 5 * ordinary + 1e-3 for t, ordinary in took.values())
