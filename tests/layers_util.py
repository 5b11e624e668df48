"""Shared by the tests of the layers: bounds, references in 64 bits and buffers.

A result is held to a bound per element, made of what its definition allows:
half a step of its own rounding, half a step of each rounded operand times the
sum of the absolute products it enters, and fp32 summation (2^-24 for each
term, relative to the sum of absolute products)."""
from __future__ import annotations

import torch

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}  # smallest subnormal
F32 = 2.0 ** -24


def poisoned(shape, dtype, dev, ld=None):
    """A tensor of all-ones bytes (NaN); with ld its rows are columns 8 .. of a
    wider tensor of that many values a row, returned too."""
    if ld is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        t.view(torch.uint8).fill_(0xFF)
        return t
    width = 1
    for s in shape[1:]:
        width *= s
    assert ld >= width + 8
    whole = torch.empty((shape[0], ld), dtype=dtype, device=dev)
    whole.view(torch.uint8).fill_(0xFF)
    return whole[:, 8:8 + width].unflatten(1, shape[1:]) if len(shape) > 2 else whole[:, 8:8 + width], whole


def spaced(t, ld):
    """t's rows as columns 8 .. of rows of ld values, NaN around them."""
    v, whole = poisoned(tuple(t.shape), t.dtype, t.device, ld)
    v.copy_(t)
    return v


def around_untouched(whole, width):
    """Nothing outside the columns 8 .. 8 + width was written."""
    b = whole.view(torch.uint8).reshape(whole.shape[0], -1)
    e = whole.element_size()
    return bool((b[:, :8 * e] == 0xFF).all()) and bool((b[:, (8 + width) * e:] == 0xFF).all())


def check(name, got, want, bound):
    """|got - want| <= bound everywhere (want, bound in 64 bits), with the worst
    excess in the message; where want is not finite, got is the same."""
    got = got.double().to(want.device)
    fine = torch.isfinite(want)
    same = torch.where(fine, torch.zeros_like(want, dtype=torch.bool),
                       (got == want) | (torch.isnan(got) & torch.isnan(want)))
    off = (got - want).abs()
    ok = torch.where(fine, off <= bound, same)
    if not bool(ok.all()):
        bad = (~ok).nonzero()
        at = tuple(bad[0].tolist())
        raise AssertionError(f"{name}: {bad.shape[0]} of {ok.numel()} outside their bounds, first at {at}: "
                             f"got {got[at].item()!r}, want {want[at].item()!r}, bound {bound[at].item():.3g}")


def rounded(t, dtype):
    """The bound's part for the output's own rounding."""
    return HALF_STEP[dtype] * t.abs() + TINY[dtype]
