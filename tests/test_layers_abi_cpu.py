"""The C entry points of the layers around the gate refuse every invalid call on
the host, before any HIP call: device addresses here are made up, so a call
that were let through would be a bug.  No GPU is needed."""
from __future__ import annotations

import ctypes
import math

import pytest

import memory_bound_engram_amd as eg
from memory_bound_engram_amd import layers

BASE = 1 << 40  # made up, 16-byte aligned, never dereferenced
BF16, FP16, FP32 = layers.BF16, layers.FP16, layers.FP32


class Call:
    """One entry point with valid arguments: pointers with their extent in
    bytes (laid one behind the other), then the rest by name."""

    def __init__(self, name, pointers, rest, order):
        self.name, self.order = name, order
        self.sizes = dict(pointers)
        self.args = dict(rest)
        at = BASE
        for p, size in pointers:
            self.args[p] = at
            at += (size + 4096) // 16 * 16

    def __call__(self, **changed):
        a = {**self.args, **changed}
        return getattr(eg.lib, self.name)(*[a[n] for n in self.order], None)


def linear_fwd(N=8, K=64, M=128, dtype=BF16, act=2):
    ws = layers.engram_linear_fwd_workspace_bytes(N, K, M)
    p = [("x", N * K * 2), ("w", M * K * 2), ("bias", M * 4), ("residual", N * M * 2), ("y", N * M * 2), ("z", N * M * 2),
         ("workspace", ws)]
    rest = dict(N=N, K=K, M=M, ldx=K, ldr=M, ldy=M, ldz=M, dtype=dtype, act=act)
    return Call("engram_linear_fwd", p, rest, [n for n, _ in p] + list(rest))


def linear_bwd(N=8, K=64, M=128, dtype=BF16, act=2):
    ws = layers.engram_linear_bwd_workspace_bytes(N, K, M)
    p = [("grad_y", N * M * 2), ("x", N * K * 2), ("w", M * K * 2), ("z", N * M * 2), ("grad_x", N * K * 2),
         ("grad_w", M * K * 2), ("grad_bias", M * 4), ("workspace", ws)]
    rest = dict(N=N, K=K, M=M, ldgy=M, ldx=K, ldz=M, ldgx=K, dtype=dtype, act=act)
    return Call("engram_linear_bwd", p, rest, [n for n, _ in p] + list(rest))


def qk_fwd(N=8, Hq=3, Hk=2, D=64, R=32, dtype=BF16):
    e = 4 if dtype == FP32 else 2
    p = [("q", N * Hq * D * e), ("k", N * Hk * D * e), ("wq", D * 4), ("wk", D * 4), ("positions", N * 8), ("freqs", R * 4),
         ("q_out", N * Hq * D * e), ("k_out", N * Hk * D * e)]
    rest = dict(N=N, Hq=Hq, Hk=Hk, D=D, R=R, ldq=Hq * D, ldk=Hk * D, ldq_out=Hq * D, ldk_out=Hk * D, eps=1e-6,
                interleaved=0, dtype=dtype)
    return Call("engram_qk_norm_rope_fwd", p, rest, [n for n, _ in p] + list(rest))


def qk_bwd(N=8, Hq=3, Hk=2, D=64, R=32, dtype=BF16):
    e = 4 if dtype == FP32 else 2
    q, k = N * Hq * D * e, N * Hk * D * e
    p = [("grad_q_out", q), ("grad_k_out", k), ("q", q), ("k", k), ("wq", D * 4), ("wk", D * 4), ("positions", N * 8),
         ("freqs", R * 4), ("grad_q", q), ("grad_k", k), ("grad_wq", D * 4), ("grad_wk", D * 4),
         ("workspace", layers.engram_qk_norm_rope_bwd_workspace_bytes(N, Hq, Hk, D))]
    rest = dict(N=N, Hq=Hq, Hk=Hk, D=D, R=R, ldgq_out=Hq * D, ldgk_out=Hk * D, ldq=Hq * D, ldk=Hk * D, ldgq=Hq * D,
                ldgk=Hk * D, eps=1e-6, interleaved=0, dtype=dtype)
    return Call("engram_qk_norm_rope_bwd", p, rest, [n for n, _ in p] + list(rest))


def decay_fwd(N=100, B=2, H=3, Dk=64, Dv=32):
    k, v, s = N * H * Dk * 2, N * H * Dv * 2, B * H * Dk * Dv * 4
    p = [("q", k), ("k", k), ("v", v), ("log_decay", H * 4), ("cu_seqlens", (B + 1) * 8), ("state_in", s), ("o", v),
         ("state_out", s), ("workspace", layers.engram_decay_attn_fwd_workspace_bytes(N, B, H, Dk, Dv))]
    rest = dict(N=N, B=B, H=H, Dk=Dk, Dv=Dv, ldq=H * Dk, ldk=H * Dk, ldv=H * Dv, ldo=H * Dv, scale=0.5)
    return Call("engram_decay_attn_fwd", p, rest, [n for n, _ in p] + list(rest))


def decay_bwd(N=100, B=2, H=3, Dk=64, Dv=32):
    k, v, s = N * H * Dk * 2, N * H * Dv * 2, B * H * Dk * Dv * 4
    p = [("grad_o", v), ("q", k), ("k", k), ("v", v), ("log_decay", H * 4), ("cu_seqlens", (B + 1) * 8), ("state_in", s),
         ("grad_state_out", s), ("grad_q", k), ("grad_k", k), ("grad_v", v), ("grad_state_in", s),
         ("workspace", layers.engram_decay_attn_bwd_workspace_bytes(N, B, H, Dk, Dv))]
    rest = dict(N=N, B=B, H=H, Dk=Dk, Dv=Dv, ldgo=H * Dv, ldq=H * Dk, ldk=H * Dk, ldv=H * Dv, ldgq=H * Dk, ldgk=H * Dk,
                ldgv=H * Dv, scale=0.5)
    return Call("engram_decay_attn_bwd", p, rest, [n for n, _ in p] + list(rest))


def decay_step(B=8, H=3, Dk=64, Dv=32, slots_total=5):
    k, v = B * H * Dk * 2, B * H * Dv * 2
    p = [("q", k), ("k", k), ("v", v), ("log_decay", H * 4), ("state", slots_total * H * Dk * Dv * 4), ("slots", B * 8),
         ("o", v)]
    rest = dict(B=B, H=H, Dk=Dk, Dv=Dv, slots_total=slots_total, ldq=H * Dk, ldk=H * Dk, ldv=H * Dv, ldo=H * Dv, scale=0.5)
    return Call("engram_decay_attn_step", p, rest, [n for n, _ in p] + list(rest))


CALLS = dict(linear_fwd=linear_fwd, linear_bwd=linear_bwd, qk_fwd=qk_fwd, qk_bwd=qk_bwd, decay_fwd=decay_fwd,
             decay_bwd=decay_bwd, decay_step=decay_step)
OPTIONAL = dict(linear_fwd={"bias", "residual", "z"}, linear_bwd={"grad_x", "grad_w", "grad_bias"}, qk_fwd=set(),
                qk_bwd=set(), decay_fwd={"state_in", "state_out"},
                decay_bwd={"state_in", "grad_state_out", "grad_state_in"}, decay_step=set())
OUTPUTS = dict(linear_fwd=["y", "z", "workspace"], linear_bwd=["grad_x", "grad_w", "grad_bias", "workspace"],
               qk_fwd=["q_out", "k_out"], qk_bwd=["grad_q", "grad_k", "grad_wq", "grad_wk", "workspace"],
               decay_fwd=["o", "state_out", "workspace"],
               decay_bwd=["grad_q", "grad_k", "grad_v", "grad_state_in", "workspace"], decay_step=["o", "state"])
INT64S = {"positions", "freqs", "cu_seqlens", "slots"}  # need 8 bytes of alignment, all others 16


def make(name):
    c = CALLS[name]()
    if name == "linear_fwd":  # of a size whose contraction is split
        c = linear_fwd(N=200, K=4096, M=256)
        assert c.sizes["workspace"] > 0
    return c


@pytest.mark.parametrize("name", CALLS)
def test_null_pointers(name):
    c = make(name)
    for p in c.sizes:
        if p not in OPTIONAL[name]:
            assert c(**{p: None}) == eg.ERR_NULL, p


def test_null_pointers_that_depend():
    c = linear_bwd()
    assert c(grad_x=None, grad_w=None, grad_bias=None) == eg.ERR_NULL
    # without an activation z is not looked at: the call is refused for what is wrong besides
    assert linear_bwd(act=0)(z=None, N=0) == eg.ERR_N_RANGE
    assert linear_bwd(act=0)(z=BASE + 2, N=0) == eg.ERR_N_RANGE
    # without a rotation neither are its arrays
    for make_qk in (qk_fwd, qk_bwd):
        assert make_qk()(R=0, positions=None, freqs=None, N=0) == eg.ERR_N_RANGE
    assert linear_fwd()(workspace=None, N=0) == eg.ERR_N_RANGE  # (8 x 64 x 128 needs no workspace)


@pytest.mark.parametrize("name", CALLS)
def test_misaligned_pointers(name):
    c = make(name)
    for p in c.sizes:
        assert c(**{p: c.args[p] + (4 if p in INT64S else 8)}) == eg.ERR_ALIGN, p
    for p in INT64S & set(c.sizes):  # 8 bytes are enough there: the call then fails for the other argument
        other = "y" if "y" in c.sizes else "q"
        assert c(**{p: c.args[p] + 8, other: c.args[other] + 2}) == eg.ERR_ALIGN


LIMITS = dict(
    linear=dict(N=layers.LINEAR_ROWS_MAX, K=layers.LINEAR_WIDTH_MAX, M=layers.LINEAR_WIDTH_MAX),
    qk=dict(N=layers.QK_ROWS_MAX, Hq=layers.QK_HEADS_MAX, Hk=layers.QK_HEADS_MAX, D=layers.QK_D_MAX),
    decay=dict(N=layers.DECAY_ROWS_MAX, B=layers.DECAY_STATES_MAX // 3, H=layers.DECAY_HEADS_MAX, Dk=layers.DECAY_D_MAX,
               Dv=layers.DECAY_D_MAX))


@pytest.mark.parametrize("name", CALLS)
def test_sizes_out_of_range(name):
    c = make(name)
    limits = dict(LIMITS[name.split("_")[0]])
    if name == "decay_step":
        limits.pop("N")
        limits["B"] = layers.DECAY_STEP_ROWS_MAX
    for size, most in limits.items():
        for v in (0, -1, -8, most + 8, 1 << 40, -(1 << 63), (1 << 63) - 1):
            assert c(**{size: v}) == eg.ERR_N_RANGE, (size, v)


def test_states_out_of_range():
    assert decay_fwd()(B=layers.DECAY_STATES_MAX // 3 + 1) == eg.ERR_N_RANGE
    for v in (0, -1, 1 << 60, (1 << 63) - 1):
        assert decay_step()(slots_total=v) == eg.ERR_N_RANGE


@pytest.mark.parametrize("name", CALLS)
def test_leading_dimensions(name):
    c = make(name)
    for ld in [n for n in c.order if n.startswith("ld")]:
        width = c.args[ld]
        for v in (width - 8, 0, -width, layers.LD_MAX + 8, 1 << 60):
            assert c(**{ld: v}) == eg.ERR_N_RANGE, (ld, v)
        assert c(**{ld: width + 4}) == eg.ERR_ALIGN, ld


@pytest.mark.parametrize("name", CALLS)
def test_widths_that_are_no_multiple_of_eight(name):
    c = make(name)
    for size in {"K", "M", "D", "Dk", "Dv"} & set(c.order):
        assert c(**{size: c.args[size] - 4, **{ld: c.args[ld] for ld in c.order if ld.startswith("ld")}}) == eg.ERR_ALIGN
    if "R" in c.order:
        assert c(R=24) == eg.ERR_ALIGN
        for v in (-16, 80, 1 << 40):
            assert c(R=v) == eg.ERR_N_RANGE


@pytest.mark.parametrize("name", CALLS)
def test_scalars(name):
    c = make(name)
    if "eps" in c.order:
        for v in (-1e-9, 1.5, math.inf, math.nan):
            assert c(eps=v) == eg.ERR_N_RANGE
    if "scale" in c.order:
        for v in (math.inf, -math.inf, math.nan):
            assert c(scale=v) == eg.ERR_N_RANGE
    if "dtype" in c.order:
        for v in (-1, 3, 1 << 20) + ((FP32,) if "act" in c.order else ()):
            assert c(dtype=v) == eg.ERR_KIND
    if "act" in c.order:
        for v in (-1, 4):
            assert c(act=v) == eg.ERR_KIND


@pytest.mark.parametrize("name", CALLS)
def test_outputs_overlap_nothing(name):
    c = make(name)
    for out in OUTPUTS[name]:
        for p, size in c.sizes.items():
            if p == out or size == 0:
                continue
            assert c(**{out: c.args[p]}) == eg.ERR_OVERLAP, (out, p)
            last = (c.args[p] + size - 1) // 16 * 16  # only the last bytes met
            assert c(**{out: last}) == eg.ERR_OVERLAP, (out, p)


def test_columns_of_packed_rows_are_apart():
    """An output may be columns of the rows that hold the inputs, but not one
    value of the same columns.  (Valid placements are refused for eps alone.)"""
    N, Hq, Hk, D, ld = 8, 3, 2, 64, 1024
    c = qk_fwd(N, Hq, Hk, D)
    lds = dict(ldq=ld, ldk=ld, ldq_out=ld, ldk_out=ld)
    row = c.args["q"] + (1 << 30)
    cols = dict(q=row, k=row + 192 * 2, q_out=row + 320 * 2, k_out=row + 512 * 2)  # 192 + 128 + 192 + 128 values
    bad_scale = dict(eps=2.0)
    assert c(**cols, **lds, **bad_scale) == eg.ERR_N_RANGE
    for out, at in (("q_out", 312), ("q_out", 328), ("k_out", 504), ("q_out", 0), ("k_out", 1024 - 64)):
        moved = dict(cols, **{out: row + at * 2})
        assert c(**moved, **lds) == eg.ERR_OVERLAP, (out, at)
    # other leading dimensions over the same bytes meet somewhere
    assert c(**cols, **dict(lds, ldq_out=ld + 8)) == eg.ERR_OVERLAP


def test_inputs_may_share_memory():
    c = decay_fwd(Dk=64, Dv=64)
    assert c(k=c.args["q"], v=c.args["q"], scale=math.nan) == eg.ERR_N_RANGE  # refused for the scale alone
    assert c(k=c.args["q"], v=c.args["q"], o=c.args["q"]) == eg.ERR_OVERLAP


def test_workspace_bytes():
    for f, good, bad in (
            (layers.engram_linear_fwd_workspace_bytes, (13, 5120, 1368), [(0, 64, 64), (4, 60, 64), (4, 64, 4), (4, 64, 1 << 40)]),
            (layers.engram_linear_bwd_workspace_bytes, (13, 5120, 1368), [(0, 64, 64), (4, 60, 64), (1 << 40, 64, 64)]),
            (layers.engram_qk_norm_rope_bwd_workspace_bytes, (8, 3, 2, 64), [(0, 3, 2, 64), (8, 0, 2, 64), (8, 3, 2, 60)]),
            (layers.engram_decay_attn_fwd_workspace_bytes, (100, 2, 3, 64, 32),
             [(0, 2, 3, 64, 32), (100, 0, 3, 64, 32), (100, 2, 3, 60, 32), (100, 2, 3, 64, 136)]),
            (layers.engram_decay_attn_bwd_workspace_bytes, (100, 2, 3, 64, 32), [(100, 2, 0, 64, 32), (100, 2, 3, 64, 0)])):
        assert f(*good) >= 0
        for sizes in bad:
            assert f(*sizes) == 0, (f.__name__, sizes)
    # at the limits the sizes stay sane (no overflow): below 16 bytes for each value of the largest operand
    n, w = layers.LINEAR_ROWS_MAX, layers.LINEAR_WIDTH_MAX
    assert 0 <= layers.engram_linear_fwd_workspace_bytes(n, w, w) < 1 << 44
    assert 2 * n * w <= layers.engram_linear_bwd_workspace_bytes(n, w, w) < 1 << 44
    h = layers.DECAY_HEADS_MAX
    assert 0 < layers.engram_decay_attn_fwd_workspace_bytes(layers.DECAY_ROWS_MAX, 1, h, 128, 128) < 1 << 44


@pytest.mark.parametrize("theta,R", [(1e4, 128), (5e5, 64), (1.0, 16), (0.25, 32), (1e4, 512)])
def test_rope_freqs(theta, R):
    """Each entry is theta^(-2i/R) / (2 pi) turns to 64 bits of a turn, here to
    the 50 bits that Python's floats can tell."""
    got = layers.engram_rope_freqs(theta, R)
    assert got.shape == (R // 2,)
    for i, g in enumerate(got.tolist()):
        turn = theta ** (-2.0 * i / R) / (2.0 * math.pi) % 1.0
        off = abs((g % (1 << 64)) / 2.0 ** 64 - turn)
        assert min(off, 1.0 - off) <= 2.0 ** -50 * max(1.0, theta ** (-2.0 * i / R)), i


def test_rope_freqs_refuses():
    table = (ctypes.c_int64 * 256)()
    f = eg.lib.engram_rope_freqs
    assert f(1e4, 128, None) == eg.ERR_NULL
    for theta, R in ((0.0, 64), (-1.0, 64), (math.inf, 64), (math.nan, 64), (1e4, 0), (1e4, -16), (1e4, 528), (1e4, 1 << 40)):
        assert f(theta, R, table) == eg.ERR_N_RANGE
    assert f(1e4, 24, table) == eg.ERR_ALIGN
    assert list(table) == [0] * 256


def test_kind_has_a_message():
    assert eg.lib.engram_status_string(eg.ERR_KIND)
    assert str(eg.EngramError(eg.ERR_KIND))
