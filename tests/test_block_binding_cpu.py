"""The binding of the rest of a block checks tensor arguments before anything
reaches the C ABI: each case builds the arguments as meta tensors, breaks one, and
expects a ValueError that names it -- with a library that fails the test if an
entry point is called.  Correct arguments that are not on a GPU are refused too."""
from __future__ import annotations

import pytest
import torch

import memory_bound_engram_amd as eg
from test_layers_binding_cpu import _NoCalls, gpu, meta, ws

bf16, fp16, fp32, i64 = torch.bfloat16, torch.float16, torch.float32, torch.int64


@pytest.fixture(autouse=True)
def no_library_calls(monkeypatch):
    monkeypatch.setattr(eg, "lib", _NoCalls(eg.lib))


N, D, B, HQ, HK, HD, SLOTS, CAP = 300, 72, 4, 6, 3, 64, 7, 700


def norm_fwd(dt=bf16):
    return dict(x=meta((N, D), dt), w=meta((D,), fp32), y=meta((N, D), dt), b=meta((D,), fp32), saved=meta((N, 2), fp32))


def norm_bwd(dt=bf16):
    return dict(grad_y=meta((N, D), dt), x=meta((N, D), dt), w=meta((D,), fp32), saved=meta((N, 2), fp32),
                grad_x=meta((N, D), dt), workspace=ws(eg.engram_layer_norm_bwd_workspace_bytes(N, D)), grad_w=meta((D,), fp32),
                grad_b=meta((D,), fp32), grad_residual=meta((N, D), dt))


def window_fwd(dt=bf16):
    return dict(q=meta((N, HQ, HD), dt), k=meta((N, HK, HD), dt), v=meta((N, HK, HD), dt), cu_seqlens=meta((B + 1,), i64),
                o=meta((N, HQ, HD), dt), window=20, sinks=4, lse=meta((N, HQ), fp32), scale=0.125)


def window_bwd(dt=bf16):
    q, k = (N, HQ, HD), (N, HK, HD)
    return dict(grad_o=meta(q, dt), q=meta(q, dt), k=meta(k, dt), v=meta(k, dt), o=meta(q, dt), lse=meta((N, HQ), fp32),
                cu_seqlens=meta((B + 1,), i64), grad_q=meta(q, dt), grad_k=meta(k, dt), grad_v=meta(k, dt),
                workspace=ws(eg.engram_window_attn_bwd_workspace_bytes(N, B, HQ, HK, HD, 20, 4)), window=20, sinks=4,
                scale=0.125)


def window_step(dt=bf16):
    pool = (SLOTS, HK, CAP, HD)
    return dict(q=meta((B, HQ, HD), dt), k=meta((B, HK, HD), dt), v=meta((B, HK, HD), dt), cache_k=meta(pool, dt),
                cache_v=meta(pool, dt), slots=meta((B,), i64), positions=meta((B,), i64), o=meta((B, HQ, HD), dt),
                workspace=ws(eg.engram_window_attn_step_workspace_bytes(B, HQ, HK, HD, CAP)), window=600, sinks=4,
                scale=0.125)


def window_fill(dt=bf16):
    pool = (SLOTS, HK, CAP, HD)
    return dict(k=meta((N, HK, HD), dt), v=meta((N, HK, HD), dt), cu_seqlens=meta((B + 1,), i64), slots=meta((B,), i64),
                cache_k=meta(pool, dt), cache_v=meta(pool, dt), sinks=4)


def scan_fwd(dt=bf16):
    return dict(gate=meta((N, D), dt), u=meta((N, D), dt), cu_seqlens=meta((B + 1,), i64), h=meta((N, D), dt),
                workspace=ws(eg.engram_gated_scan_fwd_workspace_bytes(N, B, D)), state_in=meta((B, D), fp32),
                state_out=meta((B, D), fp32))


def scan_bwd(dt=bf16):
    r, s = (N, D), (B, D)
    return dict(grad_h=meta(r, dt), gate=meta(r, dt), u=meta(r, dt), h=meta(r, dt), cu_seqlens=meta((B + 1,), i64),
                grad_gate=meta(r, dt), grad_u=meta(r, dt), workspace=ws(eg.engram_gated_scan_bwd_workspace_bytes(N, B, D)),
                state_in=meta(s, fp32), grad_state_out=meta(s, fp32), grad_state_in=meta(s, fp32))


def scan_step(dt=bf16):
    return dict(gate=meta((B, D), dt), u=meta((B, D), dt), state=meta((SLOTS, D), fp32), slots=meta((B,), i64),
                h=meta((B, D), dt))


CALLS = {"engram_layer_norm_fwd": norm_fwd, "engram_layer_norm_bwd": norm_bwd, "engram_window_attn_fwd": window_fwd,
         "engram_window_attn_bwd": window_bwd, "engram_window_attn_step": window_step,
         "engram_window_cache_fill": window_fill, "engram_gated_scan_fwd": scan_fwd, "engram_gated_scan_bwd": scan_bwd,
         "engram_gated_scan_step": scan_step}
DENSE = {"w", "b", "saved", "lse", "cu_seqlens", "cache_k", "cache_v", "slots", "positions", "state", "state_in", "state_out",
         "grad_w", "grad_b", "grad_state_in", "grad_state_out"}
# the argument that sets the type, the sizes that an argument alone sets
FIRST = {f: "x" if "norm" in f else "gate" if "scan" in f else "k" if "fill" in f else "q" for f in CALLS}
FREE = {("cache_k", 0), ("cache_k", 2), ("state", 0)}


def tensors(f, but=()):
    return [n for n, t in CALLS[f]().items() if isinstance(t, torch.Tensor) and n not in but]


def each(*, but=()):
    return [(f, n) for f in CALLS for n in tensors(f, but)]


def on_gpu(f):
    return {n: gpu(t) if isinstance(t, torch.Tensor) else t for n, t in CALLS[f]().items()}


def refused(f, name, bad, match=None):
    a = on_gpu(f)
    a[name] = gpu(bad) if isinstance(bad, torch.Tensor) else bad
    with pytest.raises(ValueError, match=match or f"^{name}:"):
        getattr(eg, f)(**a)


@pytest.mark.parametrize("f", CALLS)
def test_correct_arguments_are_refused_only_for_their_device(f):
    with pytest.raises(ValueError, match="on meta.*GPU"):
        getattr(eg, f)(**CALLS[f]())
    with pytest.raises(AssertionError, match="reached the library"):  # and pass every check if they say they are there
        with pytest.MonkeyPatch.context() as m:
            m.setattr(eg.layers, "_device", lambda: 0)
            getattr(eg, f)(**on_gpu(f), stream=0)


@pytest.mark.parametrize("f", CALLS)
def test_cpu_tensors_are_refused(f):
    a = {n: torch.empty(t.shape, dtype=t.dtype) if isinstance(t, torch.Tensor) else t for n, t in CALLS[f]().items()}
    with pytest.raises(ValueError, match="on cpu.*GPU"):
        getattr(eg, f)(**a)


@pytest.mark.parametrize("f,name", each(but=("workspace",)))
def test_types(f, name):
    t = CALLS[f]()[name]
    for dtype in (torch.float64, torch.int32, torch.bool, fp16 if t.dtype == bf16 else bf16):
        if name == FIRST[f] and dtype == fp16:
            continue  # a type the call has: then the others are the odd ones
        refused(f, name, meta(t.shape, dtype))


@pytest.mark.parametrize("f", CALLS)
def test_one_type_for_all(f):
    t = CALLS[f]()[FIRST[f]]
    refused(f, FIRST[f], meta(t.shape, fp16), match=": dtype bfloat16, expected float16")


def test_fp32_is_no_type_of_the_attention():
    for f in CALLS:
        t = CALLS[f]()[FIRST[f]]
        if "window" in f:
            refused(f, FIRST[f], meta(t.shape, fp32))
        else:
            with pytest.raises(ValueError, match="on meta.*GPU"):
                getattr(eg, f)(**CALLS[f](fp32))


@pytest.mark.parametrize("f,name", each(but=("workspace",)))
def test_shapes(f, name):
    t = CALLS[f]()[name]
    for axis in range(t.dim()):
        if f == "engram_window_attn_fwd" and name == "cu_seqlens":
            continue  # any number of sequences goes with the rest
        if (name, axis) in FREE:
            # the size may be another; then what goes with it is refused
            if name == "cache_k":
                shape = list(t.shape)
                shape[axis] += 8
                refused(f, name, meta(shape, t.dtype), match="^cache_v: shape")
            continue
        shape = list(t.shape)
        shape[axis] += 8
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
    if name in DENSE:
        refused(f, name, meta((shape[0] * 2, *shape[1:]), t.dtype)[::2])
    elif t.dim() == 3:
        refused(f, name, meta((shape[1], shape[0], shape[2]), t.dtype).transpose(0, 1))  # heads before tokens
        refused(f, name, meta((shape[0], shape[1], shape[2] + 8), t.dtype)[:, :, 8:])  # heads apart


@pytest.mark.parametrize("f,name", each())
def test_devices(f, name):
    a = on_gpu(f)
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


def test_every_name_is_exported():
    for f in CALLS:
        assert f in eg.__all__
