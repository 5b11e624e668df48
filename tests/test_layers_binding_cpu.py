"""The binding of the layers around the gate checks tensor arguments before
anything reaches the C ABI: each case builds the arguments as meta tensors
(shapes, types and strides, no memory), breaks one, and expects a ValueError
that names it -- with a library that fails the test if an entry point is
called.  Correct arguments that are not on a GPU are refused too."""
from __future__ import annotations

import pytest
import torch

import memory_bound_engram_amd as eg

bf16, fp16, fp32, i64 = torch.bfloat16, torch.float16, torch.float32, torch.int64


class _NoCalls:
    def __init__(self, real):
        self._real = real

    def __getattr__(self, name):
        if name.endswith("workspace_bytes") or name == "engram_status_string":
            return getattr(self._real, name)

        def _fail(*a, **k):
            raise AssertionError(f"{name} reached the library with invalid arguments")
        return _fail


class _OnGpu(torch.Tensor):
    """A meta tensor that says it lies on GPU 0, so that every check is reached."""
    is_cuda = True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 40


@pytest.fixture(autouse=True)
def no_library_calls(monkeypatch):
    monkeypatch.setattr(eg, "lib", _NoCalls(eg.lib))


def meta(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta")


def gpu(t):
    return t.as_subclass(_OnGpu)


N, K, M, Hq, Hk, D, R, B, H, DK, DV, SLOTS = 300, 4096, 512, 3, 2, 64, 32, 4, 3, 64, 32, 7


def ws(need):
    return meta((need,), torch.uint8)


def linear_fwd(dt=bf16):
    return dict(x=meta((N, K), dt), w=meta((M, K), dt), y=meta((N, M), dt),
                workspace=ws(eg.engram_linear_fwd_workspace_bytes(N, K, M)), bias=meta((M,), fp32),
                residual=meta((N, M), dt), z=meta((N, M), dt))


def linear_bwd(dt=bf16):
    return dict(grad_y=meta((N, M), dt), x=meta((N, K), dt), w=meta((M, K), dt), grad_x=meta((N, K), dt),
                grad_w=meta((M, K), dt), workspace=ws(eg.engram_linear_bwd_workspace_bytes(N, K, M)), z=meta((N, M), dt),
                grad_bias=meta((M,), fp32), act="silu")


def qk_fwd(dt=bf16):
    return dict(q=meta((N, Hq, D), dt), k=meta((N, Hk, D), dt), wq=meta((D,), fp32), wk=meta((D,), fp32),
                positions=meta((N,), i64), freqs=meta((R // 2,), i64), q_out=meta((N, Hq, D), dt),
                k_out=meta((N, Hk, D), dt))


def qk_bwd(dt=bf16):
    return dict(grad_q_out=meta((N, Hq, D), dt), grad_k_out=meta((N, Hk, D), dt), q=meta((N, Hq, D), dt),
                k=meta((N, Hk, D), dt), wq=meta((D,), fp32), wk=meta((D,), fp32), positions=meta((N,), i64),
                freqs=meta((R // 2,), i64), grad_q=meta((N, Hq, D), dt), grad_k=meta((N, Hk, D), dt),
                grad_wq=meta((D,), fp32), grad_wk=meta((D,), fp32),
                workspace=ws(eg.engram_qk_norm_rope_bwd_workspace_bytes(N, Hq, Hk, D)))


def decay_fwd(dt=bf16):
    return dict(q=meta((N, H, DK), dt), k=meta((N, H, DK), dt), v=meta((N, H, DV), dt), log_decay=meta((H,), fp32),
                cu_seqlens=meta((B + 1,), i64), o=meta((N, H, DV), dt),
                workspace=ws(eg.engram_decay_attn_fwd_workspace_bytes(N, B, H, DK, DV)),
                state_in=meta((B, H, DK, DV), fp32), state_out=meta((B, H, DK, DV), fp32))


def decay_bwd(dt=bf16):
    return dict(grad_o=meta((N, H, DV), dt), q=meta((N, H, DK), dt), k=meta((N, H, DK), dt), v=meta((N, H, DV), dt),
                log_decay=meta((H,), fp32), cu_seqlens=meta((B + 1,), i64), grad_q=meta((N, H, DK), dt),
                grad_k=meta((N, H, DK), dt), grad_v=meta((N, H, DV), dt),
                workspace=ws(eg.engram_decay_attn_bwd_workspace_bytes(N, B, H, DK, DV)),
                state_in=meta((B, H, DK, DV), fp32), grad_state_out=meta((B, H, DK, DV), fp32),
                grad_state_in=meta((B, H, DK, DV), fp32))


def decay_step(dt=bf16):
    return dict(q=meta((B, H, DK), dt), k=meta((B, H, DK), dt), v=meta((B, H, DV), dt), log_decay=meta((H,), fp32),
                state=meta((SLOTS, H, DK, DV), fp32), slots=meta((B,), i64), o=meta((B, H, DV), dt))


CALLS = {"engram_linear_fwd": linear_fwd, "engram_linear_bwd": linear_bwd, "engram_qk_norm_rope_fwd": qk_fwd,
         "engram_qk_norm_rope_bwd": qk_bwd, "engram_decay_attn_fwd": decay_fwd, "engram_decay_attn_bwd": decay_bwd,
         "engram_decay_attn_step": decay_step}
ROWS = {"x", "y", "residual", "z", "grad_y", "grad_x", "q", "k", "q_out", "k_out", "grad_q_out", "grad_k_out", "grad_q",
        "grad_k", "v", "o", "grad_o", "grad_v"}  # may have their rows apart
FIRST = {"engram_linear_fwd": "x", "engram_linear_bwd": "x", "engram_qk_norm_rope_fwd": "q", "engram_qk_norm_rope_bwd": "q",
         "engram_decay_attn_fwd": "q", "engram_decay_attn_bwd": "q", "engram_decay_attn_step": "q"}  # sets N


def each(*, but=()):
    return [(f, n) for f, make in CALLS.items() for n, t in make().items() if isinstance(t, torch.Tensor) and n not in but]


@pytest.mark.parametrize("f", CALLS)
def test_correct_arguments_are_refused_only_for_their_device(f):
    with pytest.raises(ValueError, match="on meta.*GPU"):
        getattr(eg, f)(**CALLS[f]())
    with pytest.raises(AssertionError, match="reached the library"):  # and pass every check if they say they are there
        with pytest.MonkeyPatch.context() as m:
            m.setattr(eg.layers, "_device", lambda: 0)
            getattr(eg, f)(**{n: gpu(t) if isinstance(t, torch.Tensor) else t for n, t in CALLS[f]().items()}, stream=0)


@pytest.mark.parametrize("f", CALLS)
def test_cpu_tensors_are_refused(f):
    a = {n: torch.empty(t.shape, dtype=t.dtype) if isinstance(t, torch.Tensor) else t for n, t in CALLS[f]().items()}
    with pytest.raises(ValueError, match="on cpu.*GPU"):
        getattr(eg, f)(**a)


def refused(f, name, bad, match=None):
    a = {n: gpu(t) if isinstance(t, torch.Tensor) else t for n, t in CALLS[f]().items()}
    a[name] = gpu(bad) if isinstance(bad, torch.Tensor) else bad
    with pytest.raises(ValueError, match=match or f"^{name}:"):
        getattr(eg, f)(**a)


@pytest.mark.parametrize("f,name", each(but=("workspace",)))
def test_types(f, name):
    t = CALLS[f]()[name]
    for dtype in (torch.float64, torch.int32, torch.bool, fp16 if t.dtype == bf16 else bf16):
        if name == FIRST[f] and dtype == fp16 and "decay" not in f:
            continue  # a type the call has: then the others are the odd ones
        refused(f, name, meta(t.shape, dtype))


@pytest.mark.parametrize("f", [f for f in CALLS if "decay" not in f])
def test_one_type_for_all(f):
    first = FIRST[f]
    t = CALLS[f]()[first]
    refused(f, first, meta(t.shape, fp16), match=": dtype bfloat16, expected float16")


def test_fp32_is_a_type_of_the_norm_alone():
    refused("engram_linear_fwd", "x", meta((N, K), fp32))
    refused("engram_decay_attn_fwd", "q", meta((N, H, DK), fp32))
    with pytest.raises(ValueError, match="on meta.*GPU"):
        eg.engram_qk_norm_rope_fwd(**qk_fwd(fp32))


@pytest.mark.parametrize("f,name", each(but=("workspace",)))
def test_shapes(f, name):
    t = CALLS[f]()[name]
    for axis in range(t.dim()):
        if (name, axis) in {("freqs", 0), ("state", 0)}:
            continue  # sets a size that no other tensor shares
        shape = list(t.shape)
        shape[axis] += 8
        # the size may be one that this tensor sets: then another is refused against it
        refused(f, name, meta(shape, t.dtype), match="shape|needs|none given")
    for shape in (t.shape[1:], (1, *t.shape)):
        refused(f, name, meta(shape, t.dtype), match=f"^{name}: (shape|.*dimensions)")


@pytest.mark.parametrize("f,name", each(but=("workspace",)))
def test_layouts(f, name):
    t = CALLS[f]()[name]
    if t.dim() == 1:
        refused(f, name, meta((2 * t.shape[0],), t.dtype)[::2])
        refused(f, name, meta((1,), t.dtype).expand(t.shape))
        return
    shape = tuple(t.shape)
    refused(f, name, meta((*shape[:-1], 2 * shape[-1]), t.dtype)[..., ::2])  # every other value
    refused(f, name, meta((1, *shape[1:]), t.dtype).expand(shape))  # one row for all
    refused(f, name, meta((*shape[:-2], shape[-1], shape[-2]), t.dtype).transpose(-1, -2))
    if name not in ROWS:
        refused(f, name, meta((shape[0] * 2, *shape[1:]), t.dtype)[::2])
    if t.dim() == 3:
        refused(f, name, meta((shape[1], shape[0], shape[2]), t.dtype).transpose(0, 1))  # heads before tokens
        refused(f, name, meta((shape[0], shape[1], shape[2] + 8), t.dtype)[:, :, 8:])  # heads apart


@pytest.mark.parametrize("f,name", each())
def test_devices(f, name):
    a = {n: gpu(t) if isinstance(t, torch.Tensor) else t for n, t in CALLS[f]().items()}
    a[name] = CALLS[f]()[name]
    with pytest.raises(ValueError, match=f"^{name}: on meta"):
        getattr(eg, f)(**a)


@pytest.mark.parametrize("f", [f for f, make in CALLS.items() if "workspace" in make()])
def test_workspaces(f):
    t = CALLS[f]()["workspace"]
    assert t.shape[0] > 0
    refused(f, "workspace", meta((t.shape[0] - 1,), torch.uint8))
    refused(f, "workspace", None)
    refused(f, "workspace", meta((2 * t.shape[0],), torch.uint8)[::2])


def test_what_goes_together():
    refused("engram_linear_bwd", "z", None)
    refused("engram_linear_fwd", "act", "tanh")
    refused("engram_linear_bwd", "act", None)
    refused("engram_qk_norm_rope_fwd", "positions", None)
    refused("engram_qk_norm_rope_bwd", "positions", None)
