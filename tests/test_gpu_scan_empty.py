"""The gated recurrence over batches in which nearly all sequences are empty: their
states go through unchanged, the others are as without them, and the call takes no
longer than its bytes and a launch let it (a walk from one empty sequence to the next
takes hundreds of milliseconds here)."""
from __future__ import annotations

import time

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import poisoned
from test_gpu_gated_scan import backward, case, forward

pytestmark = pytest.mark.gpu
BF, F4 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F4], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [8, 264])
@pytest.mark.parametrize("runs", [[(0, 5), (9000, 3)], [(9000, 1), (1, 1), (70, 700), (0, 300)], [(1, 1)] * 3 + [(5000, 40)], [(9000, 0)]],
                         ids=["first", "between", "last", "none"])
def test_between_empty_ones(gpu, runs, d, dtype):
    """`runs`: so many empty sequences, then one of so many tokens; empty ones last."""
    lens = [n for empty, tokens in runs for n in [0] * empty + [tokens]] + [0] * 777
    c = case(lens, d, dtype, gpu, True, tail=2, seed=d)
    full = [i for i, n in enumerate(lens) if n]
    few = {**c, "lens": [lens[i] for i in full] or [0], "b": max(1, len(full))}
    pick = full or [0]
    few["s0"], few["ds"] = c["s0"][pick].contiguous(), c["ds"][pick].contiguous()
    few["cu"] = torch.tensor([0] + few["lens"], device=gpu).cumsum(0)
    empty = torch.tensor([n == 0 for n in lens], device=gpu)
    m = sum(lens)
    h, out = forward(c, gpu)
    h2, out2 = forward(few, gpu)
    assert torch.equal(h[:m], h2[:m]) and torch.isnan(h[m:]).all()
    assert torch.equal(out[pick], out2) and torch.equal(out[empty], c["s0"][empty])
    got, want = backward(c, h, gpu), backward(few, h, gpu)
    for g, w in zip(got[:2], want[:2]):
        assert torch.equal(g[:m], w[:m]) and torch.isnan(g[m:]).all()
    assert torch.equal(got[2][pick], want[2]) and torch.equal(got[2][empty], c["ds"][empty])


@pytest.mark.parametrize("first", [True, False], ids=["behind", "before"])
def test_a_million_empty_sequences(gpu, first):
    b, d, n = 1 << 20, 8, 3
    cu = torch.full((b + 1,), n if first else 0, dtype=torch.int64, device=gpu)
    cu[0], cu[-1] = 0, n
    gate, u = (torch.randn((n, d), generator=torch.Generator().manual_seed(i)).to(BF).to(gpu) for i in (1, 2))
    s0, out = torch.randn((b, d), device=gpu), poisoned((b, d), F4, gpu)
    h, gg, gu, gin = (poisoned(s, t, gpu) for s, t in (((n, d), BF), ((n, d), BF), ((n, d), BF), ((b, d), F4)))
    ws = poisoned((eg.engram_gated_scan_fwd_workspace_bytes(n, b, d),), torch.uint8, gpu)

    def call():
        eg.engram_gated_scan_fwd(gate, u, cu, h, ws, state_in=s0, state_out=out)
        eg.engram_gated_scan_bwd(u, gate, u, h, cu, gg, gu, ws, state_in=s0, grad_state_out=s0, grad_state_in=gin)
        torch.cuda.synchronize()
    call()
    began = time.perf_counter()
    call()
    took = time.perf_counter() - began
    print(f"a million empty sequences: {took * 1e3:.2f} ms", flush=True)
    one = 0 if first else b - 1
    rest = torch.arange(b, device=gpu) != one
    assert torch.equal(out[rest], s0[rest]) and torch.equal(gin[rest], s0[rest])
    assert torch.isfinite(out).all() and torch.isfinite(gin).all() and torch.isfinite(h).all() and torch.isfinite(gg).all()
    assert not torch.equal(out[one], s0[one]) and not torch.equal(gin[one], s0[one])
    assert took < 0.02  # 134 MB of states are 30 us
