"""Binding of the layers around the gate: linear, qk_norm_rope, decay_attn.

Like the gate's binding, these functions only marshal: they check that every
tensor has the element type, shape, layout and device that the call will touch
(ValueError otherwise, before anything reaches the library) and hand addresses,
sizes and the current stream to the C ABI.  Outputs and workspaces are the
caller's.  A tensor of rows may have its rows apart (a column slice of a wider,
packed tensor); everything else is contiguous.
"""
from __future__ import annotations

import ctypes

import memory_bound_engram_amd as _eg

try:
    import torch as _torch
except ImportError:  # the C ABI alone
    _torch = None

_P, _I64, _INT, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float

BF16, FP16, FP32 = range(3)
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
LD_MAX = 1048576
LINEAR_ROWS_MAX, LINEAR_WIDTH_MAX = 1048576, 131072
QK_ROWS_MAX, QK_HEADS_MAX, QK_D_MAX = 4194304, 1024, 512
DECAY_ROWS_MAX, DECAY_HEADS_MAX, DECAY_STATES_MAX, DECAY_D_MAX = 16777216, 1024, 4194304, 128
DECAY_STEP_ROWS_MAX = 4096


def _declare(lib):
    for name, args in {
        "engram_linear_fwd": [_P] * 7 + [_I64] * 7 + [_INT, _INT, _P],
        "engram_linear_bwd": [_P] * 8 + [_I64] * 7 + [_INT, _INT, _P],
        "engram_qk_norm_rope_fwd": [_P] * 8 + [_I64] * 9 + [_F, _INT, _INT, _P],
        "engram_qk_norm_rope_bwd": [_P] * 13 + [_I64] * 11 + [_F, _INT, _INT, _P],
        "engram_rope_freqs": [ctypes.c_double, _I64, _P],
        "engram_decay_attn_fwd": [_P] * 9 + [_I64] * 9 + [_F, _P],
        "engram_decay_attn_bwd": [_P] * 13 + [_I64] * 12 + [_F, _P],
        "engram_decay_attn_step": [_P] * 7 + [_I64] * 9 + [_F, _P],
    }.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = _INT
    for name, n in {"engram_linear_fwd_workspace_bytes": 3, "engram_linear_bwd_workspace_bytes": 3,
                    "engram_qk_norm_rope_bwd_workspace_bytes": 4, "engram_decay_attn_fwd_workspace_bytes": 5,
                    "engram_decay_attn_bwd_workspace_bytes": 5}.items():
        getattr(lib, name).argtypes = [_I64] * n
        getattr(lib, name).restype = ctypes.c_size_t


_declare(_eg.lib)

if _torch is not None:
    _CODE = {_torch.bfloat16: BF16, _torch.float16: FP16, _torch.float32: FP32}
    _BF = (_torch.bfloat16,)
    _HALVES = (_torch.bfloat16, _torch.float16)
    _FLOATS = (_torch.bfloat16, _torch.float16, _torch.float32)
    _F32, _INTS = (_torch.float32,), (_torch.int64,)


def _raw_stream():
    """The current torch stream of a device, as an address.  torch.cuda.current_stream()
    takes 2.7 us to say the same (it makes an object), more than half of a launch."""
    raw = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
    return raw if raw is not None else lambda index: _torch.cuda.current_stream(index).cuda_stream


class _Args:
    """The tensors of one call: each is checked as it is named, all for the
    device of the first."""

    __slots__ = ("device",)

    def __init__(self):
        self.device = -1

    def _refuse(self, name, t, dtypes, shape):
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: dtype {str(t.dtype)[6:]}, expected {' or '.join(str(d)[6:] for d in dtypes)}")
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")

    def _place(self, name, t):
        """A tensor that is not known to lie with the others (a device that is no
        GPU has number -1, as this call's before its first tensor)."""
        device = t.get_device() if t.is_cuda else -1
        if device < 0:
            raise ValueError(f"{name}: on {t.device}, libengram needs GPU (HIP) tensors")
        if self.device >= 0 and device != self.device:
            raise ValueError(f"{name}: on {t.device}, other arguments on cuda:{self.device}")
        self.device = device

    def dense(self, name, t, dtypes, shape):
        if t is None:
            return None
        if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == self.device >= 0:
            return t.data_ptr()  # as it should be: the fewest questions (each costs 0.06 us)
        if t.dtype not in dtypes or t.shape != shape:
            self._refuse(name, t, dtypes, shape)
        if not t.is_contiguous():
            raise ValueError(f"{name}: libengram needs this tensor contiguous")
        self._place(name, t)
        return t.data_ptr()

    def rows(self, name, t, dtypes, shape, width):
        """Address and elements between rows of a tensor of rows: each row's
        `width` values side by side, the rows at one distance."""
        if t is None:
            return None, 0
        if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == self.device >= 0:
            return t.data_ptr(), width
        if t.dtype not in dtypes or t.shape != shape:
            self._refuse(name, t, dtypes, shape)
        ld = width
        if not t.is_contiguous():
            strides, values = t.stride(), 1
            for size, stride in zip(shape[:0:-1], strides[:0:-1]):
                if size != 1 and stride != values:
                    raise ValueError(f"{name}: the values of a row are not side by side (strides {strides})")
                values *= size
            if shape[0] > 1:
                ld = strides[0]
                if ld < width:
                    raise ValueError(f"{name}: rows overlap (strides {strides})")
        self._place(name, t)
        return t.data_ptr(), ld

    def workspace(self, t, need):
        if t is None:
            if need:
                raise ValueError(f"workspace: none given, the call needs {need} bytes")
            return None
        if t.nbytes < need:
            raise ValueError(f"workspace: {t.nbytes} bytes, the call needs {need}")
        if not t.is_contiguous():
            raise ValueError("workspace: libengram needs this tensor contiguous")
        self._place("workspace", t)
        return t.data_ptr() if need else None

    def call(self, fn, args, stream):
        """The library call with the tensors' device current and on `stream`
        (default: that device's current torch stream)."""
        index = self.device
        if index != _device():
            with _torch.cuda.device(index):
                return self.call(fn, args, stream)
        if stream is None:
            stream = _raw_stream_of(index)
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        status = fn(*args, stream)
        if status:
            raise _eg.EngramError(status)


if _torch is not None:
    _raw_stream_of = _raw_stream()
    # the tensors are there, so the runtime is up, which current_device() would see to first
    _device = getattr(_torch._C, "_cuda_getDevice", _torch.cuda.current_device)


def _shape(name, t, dims):
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name}: {len(shape)} dimensions, expected {dims}")
    return shape


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act: {act!r}, expected one of {', '.join(ACTS)}")
    return ACTS[act]


def engram_linear_fwd_workspace_bytes(N: int, K: int, M: int) -> int:
    """Scratch bytes of the linear forward (0: no workspace is needed)."""
    return int(_eg.lib.engram_linear_fwd_workspace_bytes(N, K, M))


def engram_linear_bwd_workspace_bytes(N: int, K: int, M: int) -> int:
    """Scratch bytes of the linear backward."""
    return int(_eg.lib.engram_linear_bwd_workspace_bytes(N, K, M))


def engram_linear_fwd(x, w, y, workspace=None, bias=None, residual=None, z=None, act="none", stream=None) -> None:
    """Enqueue y = act(x w^T + bias) + residual.

    x [N,K], y, residual and z [N,M] bf16 or fp16, rows may be apart; w [M,K];
    bias [M] fp32.  y is written, and z (if given) takes x w^T + bias for the
    backward of an activation.  act: "none", "relu", "silu" or "gelu" (exact).
    """
    a = _Args()
    N, K = _shape("x", x, 2)
    M = _shape("w", w, 2)[0]
    dt = (x.dtype,)
    px, ldx = a.rows("x", x, _HALVES, (N, K), K)
    pw = a.dense("w", w, dt, (M, K))
    py, ldy = a.rows("y", y, dt, (N, M), M)
    pb = a.dense("bias", bias, _F32, (M,))
    pr, ldr = a.rows("residual", residual, dt, (N, M), M)
    pz, ldz = a.rows("z", z, dt, (N, M), M)
    ws = a.workspace(workspace, _eg.lib.engram_linear_fwd_workspace_bytes(N, K, M))
    a.call(_eg.lib.engram_linear_fwd, (px, pw, pb, pr, py, pz, ws, N, K, M, ldx, ldr, ldy, ldz, _CODE[x.dtype], _act(act)), stream)


def engram_linear_bwd(grad_y, x, w, grad_x, grad_w, workspace, z=None, grad_bias=None, act="none", stream=None) -> None:
    """Enqueue the linear layer's backward: grad_x [N,K], grad_w [M,K] (each
    may be None: not wanted) and grad_bias [M] fp32 from grad_y [N,M], x, w and,
    with an activation, the forward's z.  The residual's gradient is grad_y.
    With an activation the products take its gradient in x's type, in fp16 within
    that type's range."""
    a = _Args()
    N, K = _shape("x", x, 2)
    M = _shape("w", w, 2)[0]
    dt = (x.dtype,)
    code = _act(act)
    if code and z is None:
        raise ValueError(f"z: the backward of {act} needs the forward's z")
    px, ldx = a.rows("x", x, _HALVES, (N, K), K)
    pw = a.dense("w", w, dt, (M, K))
    pg, ldgy = a.rows("grad_y", grad_y, dt, (N, M), M)
    pz, ldz = a.rows("z", z, dt, (N, M), M)
    pgx, ldgx = a.rows("grad_x", grad_x, dt, (N, K), K)
    pgw = a.dense("grad_w", grad_w, dt, (M, K))
    pgb = a.dense("grad_bias", grad_bias, _F32, (M,))
    ws = a.workspace(workspace, _eg.lib.engram_linear_bwd_workspace_bytes(N, K, M))
    a.call(_eg.lib.engram_linear_bwd, (pg, px, pw, pz, pgx, pgw, pgb, ws, N, K, M, ldgy, ldx, ldz, ldgx, _CODE[x.dtype],
           code), stream)


def engram_rope_freqs(theta: float, rotary_dim: int):
    """The rotation's table, int64 [rotary_dim / 2] on the CPU: each pair's
    turns for one position, as 64-bit fractions of a turn.  Copied to the GPU
    once, it serves every call."""
    table = (_I64 * max(1, rotary_dim // 2))()
    _eg._check(_eg.lib.engram_rope_freqs(theta, rotary_dim, table))
    return _torch.tensor(list(table), dtype=_torch.int64)


def engram_qk_norm_rope_bwd_workspace_bytes(N: int, Hq: int, Hk: int, D: int) -> int:
    """Scratch bytes of the query/key norm's backward."""
    return int(_eg.lib.engram_qk_norm_rope_bwd_workspace_bytes(N, Hq, Hk, D))


def _qk_inputs(a, q, k, wq, wk, positions, freqs):
    N, Hq, D = _shape("q", q, 3)
    Hk = _shape("k", k, 3)[1]
    dt = (q.dtype,)
    R = 0 if freqs is None else 2 * _shape("freqs", freqs, 1)[0]
    pq, ldq = a.rows("q", q, _FLOATS, (N, Hq, D), Hq * D)
    pk, ldk = a.rows("k", k, dt, (N, Hk, D), Hk * D)
    pwq, pwk = a.dense("wq", wq, _F32, (D,)), a.dense("wk", wk, _F32, (D,))
    if R and positions is None:
        raise ValueError("positions: the rotation needs them")
    pp = a.dense("positions", positions, _INTS, (N,)) if R else None
    pf = a.dense("freqs", freqs, _INTS, (R // 2,)) if R else None
    return (N, Hq, Hk, D, R), (pq, pk, pwq, pwk, pp, pf), (ldq, ldk), dt


def engram_qk_norm_rope_fwd(q, k, wq, wk, positions, freqs, q_out, k_out, eps=1e-6, interleaved=False,
                            stream=None) -> None:
    """Enqueue the per-head RMS norms of q [N,Hq,D] and k [N,Hk,D] (bf16, fp16
    or fp32, tokens may be apart) with weights wq, wk [D] fp32 and the rotation
    of the first 2 len(freqs) values of each head by positions [N] int64 (freqs
    None: no rotation).  Pairs are (i, i + R/2), or neighbours if interleaved."""
    a = _Args()
    sizes, ptrs, (ldq, ldk), dt = _qk_inputs(a, q, k, wq, wk, positions, freqs)
    N, Hq, Hk, D, _ = sizes
    pqo, ldqo = a.rows("q_out", q_out, dt, (N, Hq, D), Hq * D)
    pko, ldko = a.rows("k_out", k_out, dt, (N, Hk, D), Hk * D)
    a.call(_eg.lib.engram_qk_norm_rope_fwd, (*ptrs, pqo, pko, *sizes, ldq, ldk, ldqo, ldko, eps, int(interleaved),
           _CODE[q.dtype]), stream)


def engram_qk_norm_rope_bwd(grad_q_out, grad_k_out, q, k, wq, wk, positions, freqs, grad_q, grad_k, grad_wq, grad_wk,
                            workspace, eps=1e-6, interleaved=False, stream=None) -> None:
    """Enqueue the backward: grad_q, grad_k as q and k, grad_wq, grad_wk [D]
    fp32, from the gradients of q_out and k_out and the forward's inputs."""
    a = _Args()
    sizes, ptrs, (ldq, ldk), dt = _qk_inputs(a, q, k, wq, wk, positions, freqs)
    N, Hq, Hk, D, _ = sizes
    pgqo, ldgqo = a.rows("grad_q_out", grad_q_out, dt, (N, Hq, D), Hq * D)
    pgko, ldgko = a.rows("grad_k_out", grad_k_out, dt, (N, Hk, D), Hk * D)
    pgq, ldgq = a.rows("grad_q", grad_q, dt, (N, Hq, D), Hq * D)
    pgk, ldgk = a.rows("grad_k", grad_k, dt, (N, Hk, D), Hk * D)
    pgwq, pgwk = a.dense("grad_wq", grad_wq, _F32, (D,)), a.dense("grad_wk", grad_wk, _F32, (D,))
    ws = a.workspace(workspace, _eg.lib.engram_qk_norm_rope_bwd_workspace_bytes(N, Hq, Hk, D))
    a.call(_eg.lib.engram_qk_norm_rope_bwd, (pgqo, pgko, *ptrs, pgq, pgk, pgwq, pgwk, ws, *sizes, ldgqo, ldgko, ldq, ldk,
           ldgq, ldgk, eps, int(interleaved), _CODE[q.dtype]), stream)


def engram_decay_attn_fwd_workspace_bytes(N: int, B: int, H: int, Dk: int, Dv: int) -> int:
    """Scratch bytes of the decay attention's forward."""
    return int(_eg.lib.engram_decay_attn_fwd_workspace_bytes(N, B, H, Dk, Dv))


def engram_decay_attn_bwd_workspace_bytes(N: int, B: int, H: int, Dk: int, Dv: int) -> int:
    """Scratch bytes of the decay attention's backward."""
    return int(_eg.lib.engram_decay_attn_bwd_workspace_bytes(N, B, H, Dk, Dv))


def _decay_inputs(a, q, k, v, log_decay):
    N, H, Dk = _shape("q", q, 3)
    Dv = _shape("v", v, 3)[2]
    pq, ldq = a.rows("q", q, _BF, (N, H, Dk), H * Dk)
    pk, ldk = a.rows("k", k, _BF, (N, H, Dk), H * Dk)
    pv, ldv = a.rows("v", v, _BF, (N, H, Dv), H * Dv)
    return (N, H, Dk, Dv), (pq, pk, pv, a.dense("log_decay", log_decay, _F32, (H,))), (ldq, ldk, ldv)


def engram_decay_attn_fwd(q, k, v, log_decay, cu_seqlens, o, workspace, scale=1.0, state_in=None, state_out=None,
                          stream=None) -> None:
    """Enqueue causal linear attention with decay exp(log_decay[h]) over the
    sequences that cu_seqlens [B+1] int64 (on the GPU) cuts the tokens into.
    q, k [N,H,Dk], v, o [N,H,Dv] bf16, tokens may be apart; states
    [B,H,Dk,Dv] fp32, before and behind each sequence, both optional."""
    a = _Args()
    (N, H, Dk, Dv), ptrs, lds = _decay_inputs(a, q, k, v, log_decay)
    B = _shape("cu_seqlens", cu_seqlens, 1)[0] - 1
    pcu = a.dense("cu_seqlens", cu_seqlens, _INTS, (B + 1,))
    po, ldo = a.rows("o", o, _BF, (N, H, Dv), H * Dv)
    pin = a.dense("state_in", state_in, _F32, (B, H, Dk, Dv))
    pout = a.dense("state_out", state_out, _F32, (B, H, Dk, Dv))
    ws = a.workspace(workspace, _eg.lib.engram_decay_attn_fwd_workspace_bytes(N, B, H, Dk, Dv))
    a.call(_eg.lib.engram_decay_attn_fwd, (*ptrs, pcu, pin, po, pout, ws, N, B, H, Dk, Dv, *lds, ldo, scale), stream)


def engram_decay_attn_bwd(grad_o, q, k, v, log_decay, cu_seqlens, grad_q, grad_k, grad_v, workspace, scale=1.0,
                          state_in=None, grad_state_out=None, grad_state_in=None, stream=None) -> None:
    """Enqueue the backward: the gradients of q, k, v and (if grad_state_in is
    given) of state_in, from grad_o and (if given) grad_state_out."""
    a = _Args()
    (N, H, Dk, Dv), ptrs, lds = _decay_inputs(a, q, k, v, log_decay)
    B = _shape("cu_seqlens", cu_seqlens, 1)[0] - 1
    pcu = a.dense("cu_seqlens", cu_seqlens, _INTS, (B + 1,))
    pgo, ldgo = a.rows("grad_o", grad_o, _BF, (N, H, Dv), H * Dv)
    pgq, ldgq = a.rows("grad_q", grad_q, _BF, (N, H, Dk), H * Dk)
    pgk, ldgk = a.rows("grad_k", grad_k, _BF, (N, H, Dk), H * Dk)
    pgv, ldgv = a.rows("grad_v", grad_v, _BF, (N, H, Dv), H * Dv)
    states = (B, H, Dk, Dv)
    pin, pgout = a.dense("state_in", state_in, _F32, states), a.dense("grad_state_out", grad_state_out, _F32, states)
    pgin = a.dense("grad_state_in", grad_state_in, _F32, states)
    ws = a.workspace(workspace, _eg.lib.engram_decay_attn_bwd_workspace_bytes(N, B, H, Dk, Dv))
    a.call(_eg.lib.engram_decay_attn_bwd, (pgo, *ptrs, pcu, pin, pgout, pgq, pgk, pgv, pgin, ws, N, B, H, Dk, Dv, ldgo, *lds,
           ldgq, ldgk, ldgv, scale), stream)


def engram_decay_attn_step(q, k, v, log_decay, state, slots, o, scale=1.0, stream=None) -> None:
    """Enqueue one token for each row of a decode batch: q, k [B,H,Dk], v, o
    [B,H,Dv] bf16, rows may be apart; state [slots,H,Dk,Dv] fp32, a pool updated
    in place, slots [B] int64 each row's place in it (outside: the row is
    skipped; the same place twice: in order)."""
    a = _Args()
    (B, H, Dk, Dv), ptrs, lds = _decay_inputs(a, q, k, v, log_decay)
    total = _shape("state", state, 4)[0]
    ps = a.dense("state", state, _F32, (total, H, Dk, Dv))
    pslots = a.dense("slots", slots, _INTS, (B,))
    po, ldo = a.rows("o", o, _BF, (B, H, Dv), H * Dv)
    a.call(_eg.lib.engram_decay_attn_step, (*ptrs, ps, pslots, po, B, H, Dk, Dv, total, *lds, ldo, scale), stream)


__all__ = ["engram_linear_fwd", "engram_linear_bwd", "engram_linear_fwd_workspace_bytes",
           "engram_linear_bwd_workspace_bytes", "engram_rope_freqs", "engram_qk_norm_rope_fwd",
           "engram_qk_norm_rope_bwd", "engram_qk_norm_rope_bwd_workspace_bytes", "engram_decay_attn_fwd",
           "engram_decay_attn_bwd", "engram_decay_attn_step", "engram_decay_attn_fwd_workspace_bytes",
           "engram_decay_attn_bwd_workspace_bytes"]
