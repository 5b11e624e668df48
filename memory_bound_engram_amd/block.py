"""Binding of the rest of a block around the gate: layer_norm, window_attn, gated_scan.

In the manner of the layers' binding, whose checks it shares: every tensor's
element type, shape, layout and device is checked (ValueError otherwise, before
anything reaches the library), then addresses, sizes and the current stream go
to the C ABI.  Outputs and workspaces are the caller's; a tensor of rows may
have its rows apart.
"""
from __future__ import annotations

import ctypes

import memory_bound_engram_amd as _eg
from memory_bound_engram_amd import layers as _layers
from memory_bound_engram_amd.layers import _Args, _shape

_P, _I64, _INT, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float

NORM_ROWS_MAX, NORM_D_MAX = 2097152, 16384
WINDOW_ROWS_MAX, WINDOW_HEADS_MAX, WINDOW_HEAD_ROWS_MAX = 4194304, 1024, 536870912
WINDOW_SEQ_HEADS_MAX, WINDOW_D_MAX, WINDOW_SINKS_MAX = 1048576, 128, 128
WINDOW_STEP_ROWS_MAX, WINDOW_CAPACITY_MAX = 4096, 1048576
SCAN_ROWS_MAX, SCAN_STATES_MAX, SCAN_D_MAX, SCAN_VALUES_MAX = 16777216, 4194304, 65536, 34359738368
SCAN_STEP_ROWS_MAX = 4096


def _declare(lib):
    for name, args in {
        "engram_layer_norm_fwd": [_P] * 5 + [_I64] * 4 + [_F, _INT, _P],
        "engram_layer_norm_bwd": [_P] * 9 + [_I64] * 6 + [_INT, _P],
        "engram_window_attn_fwd": [_P] * 6 + [_I64] * 11 + [_F, _INT, _P],
        "engram_window_attn_bwd": [_P] * 11 + [_I64] * 15 + [_F, _INT, _P],
        "engram_window_attn_step": [_P] * 9 + [_I64] * 12 + [_F, _INT, _P],
        "engram_window_cache_fill": [_P] * 6 + [_I64] * 9 + [_INT, _P],
        "engram_gated_scan_fwd": [_P] * 7 + [_I64] * 6 + [_INT, _P],
        "engram_gated_scan_bwd": [_P] * 11 + [_I64] * 9 + [_INT, _P],
        "engram_gated_scan_step": [_P] * 5 + [_I64] * 6 + [_INT, _P],
    }.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = _INT
    for name, n in {"engram_layer_norm_bwd_workspace_bytes": 2, "engram_window_attn_bwd_workspace_bytes": 7,
                    "engram_window_attn_step_workspace_bytes": 5,
                    "engram_gated_scan_fwd_workspace_bytes": 3, "engram_gated_scan_bwd_workspace_bytes": 3}.items():
        getattr(lib, name).argtypes = [_I64] * n
        getattr(lib, name).restype = ctypes.c_size_t


_declare(_eg.lib)

if _layers._torch is not None:
    from memory_bound_engram_amd.layers import _CODE, _F32, _FLOATS, _HALVES, _INTS


def engram_layer_norm_fwd(x, w, y, b=None, saved=None, eps=1e-5, stream=None) -> None:
    """Enqueue y = (x - mean) rstd w + b, the norm of each row of x [N,D] (bf16,
    fp16 or fp32, rows may be apart) with w and, if given, b [D] fp32.  saved
    [N,2] fp32, if given, takes mean and rstd for the backward."""
    a = _Args()
    N, D = _shape("x", x, 2)
    dt = (x.dtype,)
    px, ldx = a.rows("x", x, _FLOATS, (N, D), D)
    pw = a.dense("w", w, _F32, (D,))
    py, ldy = a.rows("y", y, dt, (N, D), D)
    pb, ps = a.dense("b", b, _F32, (D,)), a.dense("saved", saved, _F32, (N, 2))
    a.call(_eg.lib.engram_layer_norm_fwd, (px, pw, pb, py, ps, N, D, ldx, ldy, eps, _CODE[x.dtype]), stream)


def engram_layer_norm_bwd_workspace_bytes(N: int, D: int) -> int:
    """Scratch bytes of the layer norm's backward."""
    return int(_eg.lib.engram_layer_norm_bwd_workspace_bytes(N, D))


def engram_layer_norm_bwd(grad_y, x, w, saved, grad_x, workspace, grad_w=None, grad_b=None, grad_residual=None,
                          stream=None) -> None:
    """Enqueue the backward: grad_x [N,D], to which grad_residual [N,D] is added
    if given (what reaches x past the norm), and, where given, grad_w and
    grad_b [D] fp32, from grad_y [N,D] and the forward's x, w and saved."""
    a = _Args()
    N, D = _shape("x", x, 2)
    dt = (x.dtype,)
    px, ldx = a.rows("x", x, _FLOATS, (N, D), D)
    pg, ldgy = a.rows("grad_y", grad_y, dt, (N, D), D)
    pw, ps = a.dense("w", w, _F32, (D,)), a.dense("saved", saved, _F32, (N, 2))
    pr, ldgr = a.rows("grad_residual", grad_residual, dt, (N, D), D)
    pgx, ldgx = a.rows("grad_x", grad_x, dt, (N, D), D)
    pgw, pgb = a.dense("grad_w", grad_w, _F32, (D,)), a.dense("grad_b", grad_b, _F32, (D,))
    ws = a.workspace(workspace, _eg.lib.engram_layer_norm_bwd_workspace_bytes(N, D))
    a.call(_eg.lib.engram_layer_norm_bwd, (pg, px, pw, ps, pr, pgx, pgw, pgb, ws, N, D, ldgy, ldx, ldgr, ldgx, _CODE[x.dtype]),
           stream)


def _window_inputs(a, q, k, v):
    N, Hq, D = _shape("q", q, 3)
    Hk = _shape("k", k, 3)[1]
    dt = (q.dtype,)
    pq, ldq = a.rows("q", q, _HALVES, (N, Hq, D), Hq * D)
    pk, ldk = a.rows("k", k, dt, (N, Hk, D), Hk * D)
    pv, ldv = a.rows("v", v, dt, (N, Hk, D), Hk * D)
    return (N, Hq, Hk, D), dt, (pq, pk, pv), (ldq, ldk, ldv)


def engram_window_attn_fwd(q, k, v, cu_seqlens, o, window, sinks=0, lse=None, scale=1.0, stream=None) -> None:
    """Enqueue softmax attention of each token over the last `window` tokens of
    its sequence, itself among them, and its first `sinks` ones, over the
    sequences that cu_seqlens [B+1] int64 (on the GPU) cuts the tokens into.
    q, o [N,Hq,D], k, v [N,Hk,D] bf16 or fp16, tokens may be apart, Hq a multiple
    of Hk.  lse [N,Hq] fp32, if given, takes the logarithms of the softmax's sums
    for the backward."""
    a = _Args()
    (N, Hq, Hk, D), dt, ptrs, lds = _window_inputs(a, q, k, v)
    B = _shape("cu_seqlens", cu_seqlens, 1)[0] - 1
    pcu = a.dense("cu_seqlens", cu_seqlens, _INTS, (B + 1,))
    po, ldo = a.rows("o", o, dt, (N, Hq, D), Hq * D)
    pl = a.dense("lse", lse, _F32, (N, Hq))
    a.call(_eg.lib.engram_window_attn_fwd, (*ptrs, pcu, po, pl, N, B, Hq, Hk, D, window, sinks, *lds, ldo, scale,
           _CODE[q.dtype]), stream)


def engram_window_attn_bwd_workspace_bytes(N: int, B: int, Hq: int, Hk: int, D: int, window: int, sinks: int) -> int:
    """Scratch bytes of the window attention's backward."""
    return int(_eg.lib.engram_window_attn_bwd_workspace_bytes(N, B, Hq, Hk, D, window, sinks))


def engram_window_attn_bwd(grad_o, q, k, v, o, lse, cu_seqlens, grad_q, grad_k, grad_v, workspace, window, sinks=0,
                           scale=1.0, stream=None) -> None:
    """Enqueue the backward: the gradients of q, k and v (the latter two summed
    over the query heads that read them) from grad_o and the forward's inputs, o
    and lse."""
    a = _Args()
    (N, Hq, Hk, D), dt, ptrs, lds = _window_inputs(a, q, k, v)
    B = _shape("cu_seqlens", cu_seqlens, 1)[0] - 1
    pgo, ldgo = a.rows("grad_o", grad_o, dt, (N, Hq, D), Hq * D)
    po, ldo = a.rows("o", o, dt, (N, Hq, D), Hq * D)
    pl, pcu = a.dense("lse", lse, _F32, (N, Hq)), a.dense("cu_seqlens", cu_seqlens, _INTS, (B + 1,))
    pgq, ldgq = a.rows("grad_q", grad_q, dt, (N, Hq, D), Hq * D)
    pgk, ldgk = a.rows("grad_k", grad_k, dt, (N, Hk, D), Hk * D)
    pgv, ldgv = a.rows("grad_v", grad_v, dt, (N, Hk, D), Hk * D)
    ws = a.workspace(workspace, _eg.lib.engram_window_attn_bwd_workspace_bytes(N, B, Hq, Hk, D, window, sinks))
    a.call(_eg.lib.engram_window_attn_bwd, (pgo, *ptrs, po, pl, pcu, pgq, pgk, pgv, ws, N, B, Hq, Hk, D, window, sinks,
           ldgo, *lds, ldo, ldgq, ldgk, ldgv, scale, _CODE[q.dtype]), stream)


def engram_window_attn_step_workspace_bytes(B: int, Hq: int, Hk: int, D: int, capacity: int) -> int:
    """Scratch bytes of the window attention's step (0: no workspace is needed)."""
    return int(_eg.lib.engram_window_attn_step_workspace_bytes(B, Hq, Hk, D, capacity))


def engram_window_attn_step(q, k, v, cache_k, cache_v, slots, positions, o, workspace, window, sinks=0, scale=1.0,
                            stream=None) -> None:
    """Enqueue one token for each row of a decode batch: q, o [B,Hq,D], k, v
    [B,Hk,D] bf16 or fp16, rows may be apart; cache_k, cache_v
    [slots,Hk,capacity,D], a pool of caches that take k and v, capacity at least
    sinks + window; slots, positions [B] int64 (on the GPU), each row's cache
    (outside the pool: the row is skipped) and its token's place in the sequence
    (negative: skipped).  Neighbouring rows of one slot at positions one behind
    the other are one sequence's tokens in order."""
    a = _Args()
    (B, Hq, Hk, D), dt, ptrs, lds = _window_inputs(a, q, k, v)
    total, _, capacity, _ = _shape("cache_k", cache_k, 4)
    pck = a.dense("cache_k", cache_k, dt, (total, Hk, capacity, D))
    pcv = a.dense("cache_v", cache_v, dt, (total, Hk, capacity, D))
    pslots, pp = a.dense("slots", slots, _INTS, (B,)), a.dense("positions", positions, _INTS, (B,))
    po, ldo = a.rows("o", o, dt, (B, Hq, D), Hq * D)
    ws = a.workspace(workspace, _eg.lib.engram_window_attn_step_workspace_bytes(B, Hq, Hk, D, capacity))
    a.call(_eg.lib.engram_window_attn_step, (*ptrs, pck, pcv, pslots, pp, po, ws, B, Hq, Hk, D, total, capacity, window,
           sinks, *lds, ldo, scale, _CODE[q.dtype]), stream)


def engram_window_cache_fill(k, v, cu_seqlens, slots, cache_k, cache_v, sinks=0, stream=None) -> None:
    """Enqueue the filling of caches for the steps behind a prompt: sequence b of
    k, v [N,Hk,D] (tokens may be apart), cut by cu_seqlens [B+1] int64, goes into
    cache slots[b] of cache_k, cache_v [slots,Hk,capacity,D] at positions from 0
    on, as far as its tokens can still be seen."""
    a = _Args()
    N, Hk, D = _shape("k", k, 3)
    dt = (k.dtype,)
    pk, ldk = a.rows("k", k, _HALVES, (N, Hk, D), Hk * D)
    pv, ldv = a.rows("v", v, dt, (N, Hk, D), Hk * D)
    B = _shape("cu_seqlens", cu_seqlens, 1)[0] - 1
    pcu, pslots = a.dense("cu_seqlens", cu_seqlens, _INTS, (B + 1,)), a.dense("slots", slots, _INTS, (B,))
    total, _, capacity, _ = _shape("cache_k", cache_k, 4)
    pck = a.dense("cache_k", cache_k, dt, (total, Hk, capacity, D))
    pcv = a.dense("cache_v", cache_v, dt, (total, Hk, capacity, D))
    a.call(_eg.lib.engram_window_cache_fill, (pk, pv, pcu, pslots, pck, pcv, N, B, Hk, D, total, capacity, sinks, ldk, ldv,
           _CODE[k.dtype]), stream)


def engram_gated_scan_fwd_workspace_bytes(N: int, B: int, D: int) -> int:
    """Scratch bytes of the gated recurrence's forward."""
    return int(_eg.lib.engram_gated_scan_fwd_workspace_bytes(N, B, D))


def engram_gated_scan_bwd_workspace_bytes(N: int, B: int, D: int) -> int:
    """Scratch bytes of the gated recurrence's backward."""
    return int(_eg.lib.engram_gated_scan_bwd_workspace_bytes(N, B, D))


def _scan_inputs(a, gate, u):
    N, D = _shape("gate", gate, 2)
    pg, ldg = a.rows("gate", gate, _FLOATS, (N, D), D)
    pu, ldu = a.rows("u", u, (gate.dtype,), (N, D), D)
    return N, D, (gate.dtype,), (pg, pu), (ldg, ldu)


def engram_gated_scan_fwd(gate, u, cu_seqlens, h, workspace, state_in=None, state_out=None, stream=None) -> None:
    """Enqueue h_t = f_t h_{t-1} + (1 - f_t) u_t, f = sigmoid(gate), over the
    sequences that cu_seqlens [B+1] int64 (on the GPU) cuts the tokens into.
    gate, u, h [N,D] bf16, fp16 or fp32, tokens may be apart; states [B,D] fp32,
    before and behind each sequence, both optional."""
    a = _Args()
    N, D, dt, ptrs, lds = _scan_inputs(a, gate, u)
    B = _shape("cu_seqlens", cu_seqlens, 1)[0] - 1
    pcu = a.dense("cu_seqlens", cu_seqlens, _INTS, (B + 1,))
    ph, ldh = a.rows("h", h, dt, (N, D), D)
    pin, pout = a.dense("state_in", state_in, _F32, (B, D)), a.dense("state_out", state_out, _F32, (B, D))
    ws = a.workspace(workspace, _eg.lib.engram_gated_scan_fwd_workspace_bytes(N, B, D))
    a.call(_eg.lib.engram_gated_scan_fwd, (*ptrs, pcu, pin, ph, pout, ws, N, B, D, *lds, ldh, _CODE[gate.dtype]), stream)


def engram_gated_scan_bwd(grad_h, gate, u, h, cu_seqlens, grad_gate, grad_u, workspace, state_in=None,
                          grad_state_out=None, grad_state_in=None, stream=None) -> None:
    """Enqueue the backward: the gradients of gate, u and (if grad_state_in is
    given) of state_in, from grad_h, (if given) grad_state_out and the forward's
    gate, u, h and state_in."""
    a = _Args()
    N, D, dt, ptrs, lds = _scan_inputs(a, gate, u)
    B = _shape("cu_seqlens", cu_seqlens, 1)[0] - 1
    pgh, ldgh = a.rows("grad_h", grad_h, dt, (N, D), D)
    ph, ldh = a.rows("h", h, dt, (N, D), D)
    pcu = a.dense("cu_seqlens", cu_seqlens, _INTS, (B + 1,))
    pgg, ldgg = a.rows("grad_gate", grad_gate, dt, (N, D), D)
    pgu, ldgu = a.rows("grad_u", grad_u, dt, (N, D), D)
    states = (B, D)
    pin, pgout = a.dense("state_in", state_in, _F32, states), a.dense("grad_state_out", grad_state_out, _F32, states)
    pgin = a.dense("grad_state_in", grad_state_in, _F32, states)
    ws = a.workspace(workspace, _eg.lib.engram_gated_scan_bwd_workspace_bytes(N, B, D))
    a.call(_eg.lib.engram_gated_scan_bwd, (pgh, *ptrs, ph, pcu, pin, pgout, pgg, pgu, pgin, ws, N, B, D, ldgh, *lds, ldh,
           ldgg, ldgu, _CODE[gate.dtype]), stream)


def engram_gated_scan_step(gate, u, state, slots, h, stream=None) -> None:
    """Enqueue one token for each row of a decode batch: gate, u, h [B,D], rows
    may be apart; state [slots,D] fp32, a pool updated in place, slots [B] int64
    each row's place in it (outside: the row is skipped; the same place twice:
    in order)."""
    a = _Args()
    B, D, dt, ptrs, (ldg, ldu) = _scan_inputs(a, gate, u)
    total = _shape("state", state, 2)[0]
    ps = a.dense("state", state, _F32, (total, D))
    pslots = a.dense("slots", slots, _INTS, (B,))
    ph, ldh = a.rows("h", h, dt, (B, D), D)
    a.call(_eg.lib.engram_gated_scan_step, (*ptrs, ps, pslots, ph, B, D, total, ldg, ldu, ldh, _CODE[gate.dtype]), stream)


__all__ = ["engram_layer_norm_fwd", "engram_layer_norm_bwd", "engram_layer_norm_bwd_workspace_bytes",
           "engram_window_attn_fwd", "engram_window_attn_bwd", "engram_window_attn_bwd_workspace_bytes",
           "engram_window_attn_step", "engram_window_attn_step_workspace_bytes", "engram_window_cache_fill",
           "engram_gated_scan_fwd", "engram_gated_scan_bwd", "engram_gated_scan_step",
           "engram_gated_scan_fwd_workspace_bytes", "engram_gated_scan_bwd_workspace_bytes"]
