"""The C entry points of the rest of a block (layer norm, window attention, gated
scan) refuse every invalid call on the host, before any HIP call: device
addresses here are made up, so a call that were let through would be a bug.  No
GPU is needed."""
from __future__ import annotations

import math

import pytest

import memory_bound_engram_amd as eg
from memory_bound_engram_amd import block, layers
from test_layers_abi_cpu import BASE, Call

BF16, FP16, FP32 = layers.BF16, layers.FP16, layers.FP32


def call(name, p, rest):
    return Call(name, p, rest, [n for n, _ in p] + list(rest))


def norm_fwd(N=8, D=72, dtype=BF16):
    e = 4 if dtype == FP32 else 2
    p = [("x", N * D * e), ("w", D * 4), ("b", D * 4), ("y", N * D * e), ("saved", N * 8)]
    return call("engram_layer_norm_fwd", p, dict(N=N, D=D, ldx=D, ldy=D, eps=1e-5, dtype=dtype))


def norm_bwd(N=8, D=72, dtype=BF16):
    e = 4 if dtype == FP32 else 2
    r = N * D * e
    p = [("grad_y", r), ("x", r), ("w", D * 4), ("saved", N * 8), ("grad_residual", r), ("grad_x", r), ("grad_w", D * 4),
         ("grad_b", D * 4), ("workspace", block.engram_layer_norm_bwd_workspace_bytes(N, D))]
    return call("engram_layer_norm_bwd", p, dict(N=N, D=D, ldgy=D, ldx=D, ldgr=D, ldgx=D, dtype=dtype))


def window_fwd(N=100, B=2, Hq=6, Hk=3, D=64, dtype=BF16):
    q, k = N * Hq * D * 2, N * Hk * D * 2
    p = [("q", q), ("k", k), ("v", k), ("cu_seqlens", (B + 1) * 8), ("o", q), ("lse", N * Hq * 4)]
    return call("engram_window_attn_fwd", p, dict(N=N, B=B, Hq=Hq, Hk=Hk, D=D, window=20, sinks=4, ldq=Hq * D, ldk=Hk * D,
                                                  ldv=Hk * D, ldo=Hq * D, scale=0.5, dtype=dtype))


def window_bwd(N=100, B=2, Hq=6, Hk=3, D=64, dtype=BF16):
    q, k = N * Hq * D * 2, N * Hk * D * 2
    p = [("grad_o", q), ("q", q), ("k", k), ("v", k), ("o", q), ("lse", N * Hq * 4), ("cu_seqlens", (B + 1) * 8),
         ("grad_q", q), ("grad_k", k), ("grad_v", k),
         ("workspace", block.engram_window_attn_bwd_workspace_bytes(N, B, Hq, Hk, D, 20, 4))]
    lds = {f"ld{s}": (Hk if s in ("k", "v", "gk", "gv") else Hq) * D for s in ("go", "q", "k", "v", "o", "gq", "gk", "gv")}
    return call("engram_window_attn_bwd", p, dict(N=N, B=B, Hq=Hq, Hk=Hk, D=D, window=20, sinks=4, **lds, scale=0.5,
                                                  dtype=dtype))


def window_step(B=3, Hq=6, Hk=3, D=64, slots_total=4, capacity=1000, dtype=BF16):
    q, k, c = B * Hq * D * 2, B * Hk * D * 2, slots_total * Hk * capacity * D * 2
    p = [("q", q), ("k", k), ("v", k), ("cache_k", c), ("cache_v", c), ("slots", B * 8), ("positions", B * 8), ("o", q),
         ("workspace", block.engram_window_attn_step_workspace_bytes(B, Hq, Hk, D, capacity))]
    return call("engram_window_attn_step", p,
                dict(B=B, Hq=Hq, Hk=Hk, D=D, slots_total=slots_total, capacity=capacity, window=900, sinks=4, ldq=Hq * D,
                     ldk=Hk * D, ldv=Hk * D, ldo=Hq * D, scale=0.5, dtype=dtype))


def window_fill(N=100, B=2, Hk=3, D=64, slots_total=4, capacity=24, dtype=BF16):
    k, c = N * Hk * D * 2, slots_total * Hk * capacity * D * 2
    p = [("k", k), ("v", k), ("cu_seqlens", (B + 1) * 8), ("slots", B * 8), ("cache_k", c), ("cache_v", c)]
    return call("engram_window_cache_fill", p, dict(N=N, B=B, Hk=Hk, D=D, slots_total=slots_total, capacity=capacity, sinks=4,
                                                    ldk=Hk * D, ldv=Hk * D, dtype=dtype))


def scan_fwd(N=100, B=2, D=72, dtype=BF16):
    e = 4 if dtype == FP32 else 2
    r, s = N * D * e, B * D * 4
    p = [("gate", r), ("u", r), ("cu_seqlens", (B + 1) * 8), ("state_in", s), ("h", r), ("state_out", s),
         ("workspace", block.engram_gated_scan_fwd_workspace_bytes(N, B, D))]
    return call("engram_gated_scan_fwd", p, dict(N=N, B=B, D=D, ldg=D, ldu=D, ldh=D, dtype=dtype))


def scan_bwd(N=100, B=2, D=72, dtype=BF16):
    e = 4 if dtype == FP32 else 2
    r, s = N * D * e, B * D * 4
    p = [("grad_h", r), ("gate", r), ("u", r), ("h", r), ("cu_seqlens", (B + 1) * 8), ("state_in", s), ("grad_state_out", s),
         ("grad_gate", r), ("grad_u", r), ("grad_state_in", s),
         ("workspace", block.engram_gated_scan_bwd_workspace_bytes(N, B, D))]
    return call("engram_gated_scan_bwd", p, dict(N=N, B=B, D=D, ldgh=D, ldg=D, ldu=D, ldh=D, ldgg=D, ldgu=D, dtype=dtype))


def scan_step(B=8, D=72, slots_total=5, dtype=BF16):
    e = 4 if dtype == FP32 else 2
    r = B * D * e
    p = [("gate", r), ("u", r), ("state", slots_total * D * 4), ("slots", B * 8), ("h", r)]
    return call("engram_gated_scan_step", p, dict(B=B, D=D, slots_total=slots_total, ldg=D, ldu=D, ldh=D, dtype=dtype))


CALLS = dict(norm_fwd=norm_fwd, norm_bwd=norm_bwd, window_fwd=window_fwd, window_bwd=window_bwd, window_step=window_step,
             window_fill=window_fill, scan_fwd=scan_fwd, scan_bwd=scan_bwd, scan_step=scan_step)
OPTIONAL = dict(norm_fwd={"b", "saved"}, norm_bwd={"grad_residual", "grad_w", "grad_b"}, window_fwd={"lse"}, window_bwd=set(),
                window_step=set(), window_fill=set(), scan_fwd={"state_in", "state_out"},
                scan_bwd={"state_in", "grad_state_out", "grad_state_in"}, scan_step=set())
OUTPUTS = dict(norm_fwd=["y", "saved"], norm_bwd=["grad_x", "grad_w", "grad_b", "workspace"], window_fwd=["o", "lse"],
               window_bwd=["grad_q", "grad_k", "grad_v", "workspace"], window_step=["cache_k", "cache_v", "o", "workspace"],
               window_fill=["cache_k", "cache_v"], scan_fwd=["h", "state_out", "workspace"],
               scan_bwd=["grad_gate", "grad_u", "grad_state_in", "workspace"], scan_step=["h", "state"])
INT64S = {"cu_seqlens", "slots", "positions"}  # need 8 bytes of alignment, all others 16


@pytest.mark.parametrize("name", CALLS)
def test_null_pointers(name):
    c = CALLS[name]()
    for p in c.sizes:
        if p not in OPTIONAL[name]:
            assert c(**{p: None}) == eg.ERR_NULL, p


def test_a_workspace_is_asked_for_where_lists_are_split():
    assert window_step().sizes["workspace"] > 0
    c = window_step(B=3, capacity=40)
    assert c.sizes["workspace"] == 0
    assert c(window=36, workspace=None, scale=math.nan) == eg.ERR_N_RANGE  # refused for the scale alone


@pytest.mark.parametrize("name", CALLS)
def test_misaligned_pointers(name):
    c = CALLS[name]()
    for p in c.sizes:
        assert c(**{p: c.args[p] + (4 if p in INT64S else 8)}) == eg.ERR_ALIGN, p
    other = next(p for p in c.sizes if p not in INT64S)
    for p in INT64S & set(c.sizes):  # 8 bytes are enough there: the call then fails for the other argument
        assert c(**{p: c.args[p] + 8, other: c.args[other] + 2}) == eg.ERR_ALIGN


HUGE = (1 << 40, -(1 << 63), (1 << 63) - 1)
LIMITS = dict(
    norm=dict(N=block.NORM_ROWS_MAX, D=block.NORM_D_MAX),
    window=dict(N=block.WINDOW_ROWS_MAX, B=block.WINDOW_SEQ_HEADS_MAX // 3, Hq=block.WINDOW_HEADS_MAX, Hk=6,
                D=block.WINDOW_D_MAX, sinks=block.WINDOW_SINKS_MAX),
    scan=dict(N=block.SCAN_ROWS_MAX, B=block.SCAN_STATES_MAX, D=block.SCAN_D_MAX))


@pytest.mark.parametrize("name", CALLS)
def test_sizes_out_of_range(name):
    c = CALLS[name]()
    limits = dict(LIMITS[name.split("_")[0]])
    if name in ("window_step", "window_fill"):
        limits["B"] = block.WINDOW_STEP_ROWS_MAX
    if name == "window_fill":
        limits["Hk"] = block.WINDOW_HEADS_MAX
    if name == "scan_step":
        limits["B"] = block.SCAN_STEP_ROWS_MAX
    for size, most in limits.items():
        if size not in c.order:
            continue
        for v in (-1, -8, most + 8, *HUGE) + (() if size == "sinks" else (0,)):
            assert c(**{size: v}) == eg.ERR_N_RANGE, (size, v)
    if "slots_total" in c.order:
        for v in (0, -1, 1 << 60, (1 << 63) - 1):
            assert c(slots_total=v) == eg.ERR_N_RANGE
    if "capacity" in c.order:
        for v in (0, -1, block.WINDOW_CAPACITY_MAX + 1, *HUGE):
            assert c(capacity=v) == eg.ERR_N_RANGE


def test_sizes_that_depend():
    for c in (window_fwd(), window_bwd()):
        assert c(Hk=4) == eg.ERR_N_RANGE           # Hq is no multiple
        for v in (0, -1, -(1 << 63)):
            assert c(window=v) == eg.ERR_N_RANGE
        # any window is as good as all of the past: refused for the scale alone
        assert c(window=(1 << 63) - 1, sinks=block.WINDOW_SINKS_MAX, scale=-1.0) == eg.ERR_N_RANGE
        rows = block.WINDOW_HEAD_ROWS_MAX // 1024
        assert c(N=rows + 1, Hq=1024, Hk=1, **{ld: layers.LD_MAX for ld in c.order if ld.startswith("ld")}) == eg.ERR_N_RANGE
    c = window_step()
    assert c(window=997) == eg.ERR_N_RANGE and c(window=996, sinks=5) == eg.ERR_N_RANGE and c(window=0) == eg.ERR_N_RANGE
    assert window_fill()(sinks=24) == eg.ERR_N_RANGE  # no line is left for the window
    assert scan_fwd()(N=block.SCAN_VALUES_MAX // 65536 + 1, D=65536, ldg=65536, ldu=65536, ldh=65536) == eg.ERR_N_RANGE


@pytest.mark.parametrize("name", CALLS)
def test_leading_dimensions(name):
    c = CALLS[name]()
    for ld in [n for n in c.order if n.startswith("ld")]:
        width = c.args[ld]
        for v in (width - 8, 0, -width, layers.LD_MAX + 8, 1 << 60):
            assert c(**{ld: v}) == eg.ERR_N_RANGE, (ld, v)
        assert c(**{ld: width + 4}) == eg.ERR_ALIGN, ld


def test_leading_dimensions_of_what_is_not_there_are_not_looked_at():
    assert norm_bwd()(grad_residual=None, ldgr=-1, x=BASE + 2) == eg.ERR_ALIGN


@pytest.mark.parametrize("name", CALLS)
def test_widths_that_are_no_multiple_of_eight(name):
    c = CALLS[name]()
    assert c(D=c.args["D"] - 4) == eg.ERR_ALIGN


@pytest.mark.parametrize("name", CALLS)
def test_scalars(name):
    c = CALLS[name]()
    if "eps" in c.order:
        for v in (-1e-9, 1.5, math.inf, math.nan):
            assert c(eps=v) == eg.ERR_N_RANGE
    if "scale" in c.order:
        for v in (0.0, -1.0, math.inf, -math.inf, math.nan):
            assert c(scale=v) == eg.ERR_N_RANGE
    for v in (-1, 3, 1 << 20) + ((FP32,) if "window" in name else ()):
        assert c(dtype=v) == eg.ERR_KIND


@pytest.mark.parametrize("name", ["window_fwd", "window_bwd", "window_step"])
def test_a_scale_whose_exponents_would_be_infinite(name):
    """scale log2(e) has to be finite; the largest scale is let through, up to the misaligned pointer."""
    c = CALLS[name]()
    for v in (2.0 ** 126 * (1 + 2.0 ** -23), 2.0 ** 127, 3.4e38):
        assert c(scale=v) == eg.ERR_N_RANGE, v
    assert c(scale=2.0 ** 126, q=c.args["q"] + 8) == eg.ERR_ALIGN


@pytest.mark.parametrize("name", CALLS)
def test_outputs_overlap_nothing(name):
    c = CALLS[name]()
    for out in OUTPUTS[name]:
        for p, size in c.sizes.items():
            if p == out or size == 0 or c.sizes[out] == 0:
                continue
            assert c(**{out: c.args[p]}) == eg.ERR_OVERLAP, (out, p)
            last = (c.args[p] + size - 1) // 16 * 16  # only the last bytes met
            assert c(**{out: last}) == eg.ERR_OVERLAP, (out, p)


def test_columns_of_packed_rows_are_apart():
    """An output may be columns of the rows that hold the inputs, but not one value of the same columns.  (Valid
    placements are refused for the scale alone.)"""
    c = window_fwd()
    row = c.args["q"] + (1 << 30)
    lds = dict(ldq=2048, ldk=2048, ldv=2048, ldo=2048)
    cols = dict(q=row, k=row + 384 * 2, v=row + 576 * 2, o=row + 768 * 2)  # 384 + 192 + 192 + 384 values
    assert c(**cols, **lds, scale=-1.0) == eg.ERR_N_RANGE
    for at in (760, 568, 0, 2048 - 376):
        assert c(**dict(cols, o=row + at * 2), **lds) == eg.ERR_OVERLAP, at
    c = scan_bwd()
    row = c.args["gate"] + (1 << 30)
    lds = {ld: 512 for ld in c.order if ld.startswith("ld")}
    cols = dict(gate=row, u=row + 144, grad_gate=row + 288, grad_u=row + 432)
    assert c(**cols, **lds, B=0) == eg.ERR_N_RANGE
    assert c(**dict(cols, grad_u=row + 416), **lds) == eg.ERR_OVERLAP


def test_workspace_bytes():
    for f, good, bad in (
            (block.engram_layer_norm_bwd_workspace_bytes, (8, 72), [(0, 72), (8, 0), (8, 70), (8, 1 << 40), (1 << 40, 72)]),
            (block.engram_gated_scan_fwd_workspace_bytes, (100, 2, 72), [(0, 2, 72), (100, 0, 72), (100, 2, 70), (1 << 40, 2, 72)]),
            (block.engram_gated_scan_bwd_workspace_bytes, (100, 2, 72), [(0, 2, 72), (100, 2, 0)]),
            (block.engram_window_attn_bwd_workspace_bytes, (100, 2, 6, 3, 64, 20, 4),
             [(0, 2, 6, 3, 64, 20, 4), (100, 2, 6, 4, 64, 20, 4), (100, 2, 6, 3, 60, 20, 4), (100, 2, 6, 3, 136, 20, 4),
              (100, 2, 6, 3, 64, 0, 4), (100, 2, 6, 3, 64, 20, 129)]),
            (block.engram_window_attn_step_workspace_bytes, (1, 6, 3, 64, 1000),
             [(0, 6, 3, 64, 1000), (1, 6, 4, 64, 1000), (1, 6, 3, 64, 0), (1, 6, 3, 60, 1000)])):
        assert f(*good) > 0
        for sizes in bad:
            assert f(*sizes) == 0, (f.__name__, sizes)
    # at the limits the sizes stay sane (no overflow)
    assert 0 < block.engram_layer_norm_bwd_workspace_bytes(block.NORM_ROWS_MAX, block.NORM_D_MAX) < 1 << 30
    d = block.SCAN_VALUES_MAX // block.SCAN_ROWS_MAX
    assert 0 < block.engram_gated_scan_fwd_workspace_bytes(block.SCAN_ROWS_MAX, 1, d) < 1 << 36
    n = block.WINDOW_ROWS_MAX
    assert 4 * n * 128 < block.engram_window_attn_bwd_workspace_bytes(n, 1, 128, 8, 128, 1024, 128) < 1 << 33
    # the sinks' sums are part of it where something lies behind a window
    f = block.engram_window_attn_bwd_workspace_bytes
    assert f(100, 2, 6, 3, 64, 20, 4) > f(100, 2, 6, 3, 64, 20, 0) == f(100, 2, 6, 3, 64, 100, 4)
