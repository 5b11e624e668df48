"""Gates in fp32 from shut to open: f and 1 - f, each relative to itself, through a
prompt of one token, a step and the backward.

exp2 is off by a unit in the last place (two of 2^-24), the exponent's rounding is put
back with a rounding, then 1 + t, the reciprocal (a unit in the last place) and a product:
1 + 2 + 1 + 2 + 1 = 7 units of 2^-24, within the header's 2^-21."""
from __future__ import annotations

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import F32, check, poisoned

pytestmark = pytest.mark.gpu
F4, D, B = torch.float32, 4096, 3
GATE = 7 * F32


def setup(dev):
    g = torch.Generator().manual_seed(1)
    gate = (torch.linspace(-87, 87, D)[None] + 0.01 * torch.randn((B, D), generator=g)).clamp(-87, 87)
    zero, one = torch.zeros((B, D)), 1 + torch.rand((B, D), generator=g)
    return [t.to(dev) for t in (gate, zero, one)]


def prompt(gate, u, s0, dev):
    h, out = poisoned((B, D), F4, dev), poisoned((B, D), F4, dev)
    ws = poisoned((eg.engram_gated_scan_fwd_workspace_bytes(B, B, D),), torch.uint8, dev)
    eg.engram_gated_scan_fwd(gate, u, torch.arange(B + 1, device=dev), h, ws, state_in=s0, state_out=out)
    return h, out


@pytest.mark.parametrize("kept", [True, False])
def test_one_token(gpu, kept):
    """From a state and nothing new, f alone; from no state, 1 - f alone."""
    gate, zero, one = setup(gpu)
    u, s0 = (zero, one) if kept else (one, zero)
    want = torch.sigmoid(gate.double() * (1 if kept else -1)) * one.double()
    bound = want * (GATE + 2 * F32) + 2.0 ** -126  # the product, and the sum with 0 and a state handed on
    for name, got in zip(("h", "state_out"), prompt(gate, u, s0, gpu)):
        check(name, got, want, bound)
    state, h = s0.clone(), poisoned((B, D), F4, gpu)
    eg.engram_gated_scan_step(gate, u, state, torch.arange(B, device=gpu), h)
    check("step", h, want, bound)
    check("step's state", state, want, bound)


def test_gradients(gpu):
    """Of one token from a state of 1 and u of 0: du = (1 - f) g, dgate = g f (1 - f), dstate = f g."""
    gate, zero, one = setup(gpu)
    s0 = torch.ones_like(one)
    h, _ = prompt(gate, zero, s0, gpu)
    gg, gu, gin = (poisoned((B, D), F4, gpu) for _ in range(3))
    ws = poisoned((eg.engram_gated_scan_bwd_workspace_bytes(B, B, D),), torch.uint8, gpu)
    eg.engram_gated_scan_bwd(one, gate, zero, h, torch.arange(B + 1, device=gpu), gg, gu, ws, state_in=s0, grad_state_in=gin)
    g, f, n = one.double(), torch.sigmoid(gate.double()), torch.sigmoid(-gate.double())
    check("grad_u", gu, g * n, g * n * (GATE + 2 * F32) + 2.0 ** -126)
    check("grad_state_in", gin, g * f, g * f * (GATE + 2 * F32) + 2.0 ** -126)
    check("grad_gate", gg, g * f * n, g * f * n * (2 * GATE + 4 * F32) + 2.0 ** -126)
