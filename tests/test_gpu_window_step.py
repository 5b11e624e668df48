"""The window attention's single tokens over a pool of caches, and the caches'
filling, against the definition in 64 bits over whole sequences: positions from
the first token to far round the ring, windows, sinks and spare lines, head
sizes and counts, lists split over workgroups, several tokens of one sequence
in one call, padding, infinities that have left the window."""
from __future__ import annotations

import math

import pytest
import torch

import memory_bound_engram_amd as eg
from layers_util import F32, HALF_STEP, around_untouched, check, poisoned, rounded

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


class Pool:
    """Sequences with their whole pasts, and the caches that hold what can still be seen."""

    def __init__(self, dev, slots, hq, hk, d, window, sinks, spare=0, dtype=BF, seed=0):
        self.dev, self.hq, self.hk, self.d, self.window, self.sinks, self.dtype = dev, hq, hk, d, window, sinks, dtype
        self.capacity = sinks + window + spare
        self.g = torch.Generator().manual_seed(seed)
        self.cache_k, self.cache_v = (poisoned((slots, hk, self.capacity, d), dtype, dev) for _ in range(2))
        self.past = {}  # slot: (k, v) of all its tokens, on the CPU

    def normal(self, *shape, std=1.0):
        return (std * torch.randn(shape, generator=self.g)).to(self.dtype)

    def line(self, j):
        return j if j < self.sinks else self.sinks + (j - self.sinks) % (self.capacity - self.sinks)

    def fill(self, lens, slots):
        k, v = (self.normal(sum(lens), self.hk, self.d) for _ in range(2))
        at = 0
        for n, s in zip(lens, slots):
            if 0 <= s < self.cache_k.shape[0]:
                self.past[s] = (k[at:at + n], v[at:at + n])
            at += n
        packed = torch.cat((k.flatten(1), v.flatten(1)), 1).to(self.dev)
        kk, vv = (packed[:, i * self.hk * self.d:(i + 1) * self.hk * self.d].unflatten(1, (self.hk, self.d)) for i in (0, 1))
        eg.engram_window_cache_fill(kk, vv, torch.tensor([0] + lens).cumsum(0).to(self.dev),
                                    torch.tensor(slots, device=self.dev), self.cache_k, self.cache_v, sinks=self.sinks)

    def step(self, slots, positions=None):
        """One call; the tokens join their sequences' pasts in order."""
        b, n_slots = len(slots), self.cache_k.shape[0]
        q, k, v = self.normal(b, self.hq, self.d, std=2.0), self.normal(b, self.hk, self.d), self.normal(b, self.hk, self.d)
        seen, pos = [], []
        for r, s in enumerate(slots):
            if not 0 <= s < n_slots or positions is not None and positions[r] < 0:
                seen.append(None)
                pos.append(-5 if 0 <= s < n_slots else 3)
                continue
            pk, pv = self.past.get(s, (k[:0], v[:0]))
            self.past[s] = (torch.cat((pk, k[r:r + 1])), torch.cat((pv, v[r:r + 1])))
            pos.append(len(pk))
            seen.append(s)
        snap = {r: tuple(t[:pos[r] + 1] for t in self.past[s]) for r, s in enumerate(seen) if s is not None}
        packed = torch.cat((q.flatten(1), k.flatten(1), v.flatten(1)), 1).to(self.dev)
        hq, hk, d = self.hq, self.hk, self.d
        qq, kk, vv = (packed[:, x * d:(x + y) * d].unflatten(1, (y, d)) for x, y in ((0, hq), (hq, hk), (hq + hk, hk)))
        o, whole = poisoned((b, hq, d), self.dtype, self.dev, hq * d + 16)
        need = eg.engram_window_attn_step_workspace_bytes(b, hq, hk, d, self.capacity)
        ws = poisoned((need,), torch.uint8, self.dev)
        eg.engram_window_attn_step(qq, kk, vv, self.cache_k, self.cache_v, torch.tensor(slots, device=self.dev),
                                   torch.tensor(pos, device=self.dev), o, ws, self.window, sinks=self.sinks, scale=d ** -0.5)
        torch.cuda.synchronize()
        assert around_untouched(whole, hq * d)
        self.check(q, snap, o.cpu())
        return o

    def check(self, q, snap, o):
        u = HALF_STEP[self.dtype]
        for r in range(q.shape[0]):
            if r not in snap:
                assert torch.isnan(o[r]).all()  # skipped: left as it was
                continue
            k, v = (t.double() for t in snap[r])
            p = len(k) - 1
            j = torch.arange(p + 1)
            keep = (j > p - self.window) | (j < self.sinks)
            k, v = (t[keep].repeat_interleave(self.hq // self.hk, 1) for t in (k, v))
            qr = q[r].double()
            z = torch.einsum("hd,jhd->hj", qr, k) * self.d ** -0.5
            za = torch.einsum("hd,jhd->hj", qr.abs(), k.abs()) * self.d ** -0.5
            w = torch.softmax(z, 1)
            # scores: sums of d exact products, scaled and less their maximum; the weights rounded once (to fp16 those
            # below its steps lose 2^-25 of the largest), then fp32 sums and the joins of waves and workgroups
            ez = F32 * ((self.d + 4) * za.amax(1, keepdim=True) + 4 * z.abs().amax(1, keepdim=True))
            rel = torch.expm1(2 * ez) + F32 * (keep.sum() + 64)
            want = torch.einsum("hj,jhd->hd", w, v)
            bound = torch.einsum("hj,jhd->hd", w, v.abs()) * (u * (1 + rel) + rel)
            if self.dtype is FP:
                bound = bound + 2.0 ** -25 * w.amax(1, keepdim=True) * v.abs().sum(0)
            check(f"o of row {r} at position {p}", o[r], want, bound + rounded(want, self.dtype))

    def check_caches(self):
        """Every line holds the last token that belongs there, and no other line was written."""
        for s in range(self.cache_k.shape[0]):
            k, v = self.past.get(s, (torch.zeros((0, self.hk, self.d)),) * 2)
            for cache, past in ((self.cache_k[s].cpu(), k), (self.cache_v[s].cpu(), v)):
                held = {self.line(j): j for j in range(len(past))}
                for i in range(self.capacity):
                    want = past[held[i]] if i in held else None
                    got = cache[:, i]
                    assert torch.equal(got, want) if want is not None else torch.isnan(got).all(), (s, i)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("window,sinks,spare", [(1, 0, 0), (1, 2, 0), (7, 3, 0), (32, 4, 5), (100, 0, 1), (45, 128, 0)])
def test_steps_from_the_first_token_on(gpu, window, sinks, spare, dtype):
    p = Pool(gpu, 4, 4, 2, 64, window, sinks, spare, dtype)
    p.fill([5, 0, 2 * window + sinks + 3], [2, 0, 1])
    p.check_caches()
    for i in range(6 if window > 40 else 2 * window + sinks + 4):
        print(f"window step {i} window={window} sinks={sinks} {dtype}", flush=True)
        p.step([0, 2, 1] if i % 2 else [1, 0, 2, 3])
    p.check_caches()


@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 1), (16, 1), (17, 1), (70, 2), (6, 6), (40, 8)])
@pytest.mark.parametrize("d", [8, 40, 64, 80, 128])
def test_heads(gpu, hq, hk, d):
    p = Pool(gpu, 3, hq, hk, d, 75, 3, 2, seed=d)
    p.fill([200, 10], [1, 0])
    for _ in range(2):
        print(f"window step heads {hq}/{hk} d={d}", flush=True)
        p.step([1, 0, 2])


@pytest.mark.parametrize("b", [1, 3, 64])
@pytest.mark.parametrize("window", [129, 1024, 4000])
def test_long_lists(gpu, window, b):
    """Lists split over many workgroups (few rows), some, and not at all."""
    p = Pool(gpu, b + 1, 10, 2, 128, window, 4, seed=window)
    lens = [max(1, (window + 300) * (i + 1) // b) for i in range(b)]
    p.fill(lens, list(range(b)))
    print(f"window step b={b} window={window}", flush=True)
    p.step(list(range(b)))
    p.step([b] + list(range(b)))


def test_padding_and_several_tokens_of_a_sequence(gpu):
    p = Pool(gpu, 5, 4, 2, 64, 20, 3, spare=7, seed=3)
    p.fill([50, 4, 1, 30], [0, 3, 2, 7])  # slot 7 is outside
    p.check_caches()
    p.step([0, 0, 0, -1, 3, 3, 2, 2, 2, 2, 2, 2, 2, 2, 5, 1, 1])  # eight tokens of slot 2, from its second on
    p.step([1 << 40, 0, -(1 << 62), 2])
    p.step([0, 2, 1], positions=[0, -1, 0])
    p.check_caches()


def test_sequence_goes_on_in_pieces_as_the_whole_prompt(gpu):
    """Two tokens a call through the caches: what the forward gives over all tokens at once."""
    n, hq, hk, d, window, sinks = 90, 6, 2, 128, 33, 2
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((n, h, d), generator=g).to(BF).to(gpu) for h in (hq, hk, hk))
    o = torch.empty_like(q)
    eg.engram_window_attn_fwd(q, k, v, torch.tensor([0, n], device=gpu), o, window, sinks=sinks, scale=d ** -0.5)
    ck, cv = (torch.empty((1, hk, window + sinks + 1, d), dtype=BF, device=gpu) for _ in range(2))
    eg.engram_window_cache_fill(k[:40], v[:40], torch.tensor([0, 40], device=gpu), torch.tensor([0], device=gpu), ck, cv,
                                sinks=sinks)
    ws = torch.empty(eg.engram_window_attn_step_workspace_bytes(2, hq, hk, d, window + sinks + 1), dtype=torch.uint8, device=gpu)
    row, slots = torch.empty((2, hq, d), dtype=BF, device=gpu), torch.zeros(2, dtype=torch.int64, device=gpu)
    for t in range(40, n, 2):
        eg.engram_window_attn_step(q[t:t + 2], k[t:t + 2], v[t:t + 2], ck, cv, slots, torch.tensor([t, t + 1], device=gpu), row,
                                   ws, window, sinks=sinks, scale=d ** -0.5)
        # both are within 2^-8 (weights) of the sum of |p v|, at most max |v|, and a rounding of their own
        top = v.abs().max().item()
        assert ((row.double() - o[t:t + 2].double()).abs() <= 2 * 2.0 ** -8 * top + 2.0 ** -7 * o[t:t + 2].double().abs()).all()


def test_the_same_row_twice(gpu):
    """A padded batch that repeats a row: each copy gets the row's result."""
    p = Pool(gpu, 1, 4, 2, 64, 20, 2, seed=4)
    p.fill([40], [0])
    q, k, v = p.normal(1, 4, 64).to(gpu), p.normal(1, 2, 64).to(gpu), p.normal(1, 2, 64).to(gpu)
    ck, cv = p.cache_k.clone(), p.cache_v.clone()

    def run(times):
        a, b = ck.clone(), cv.clone()
        o = torch.empty((times, 4, 64), dtype=BF, device=gpu)
        ws = torch.empty(eg.engram_window_attn_step_workspace_bytes(times, 4, 2, 64, 22), dtype=torch.uint8, device=gpu)
        eg.engram_window_attn_step(q.repeat(times, 1, 1), k.repeat(times, 1, 1), v.repeat(times, 1, 1), a, b,
                                   torch.zeros(times, dtype=torch.int64, device=gpu),
                                   torch.full((times,), 40, device=gpu), o, ws, 20, sinks=2, scale=0.125)
        return o, a, b
    (o1, a1, b1), (o3, a3, b3) = run(1), run(3)
    assert all(torch.equal(o1[0], o3[i]) for i in range(3)) and torch.equal(a1, a3) and torch.equal(b1, b3)


def test_fill_with_a_slot_twice_and_bad_bounds(gpu):
    p = Pool(gpu, 3, 2, 1, 8, 10, 2, seed=5)
    p.fill([30, 5, 9], [1, 1, 0])  # the last sequence of slot 1 counts, its lines alone are written
    p.check_caches()
    k = torch.randn((6, 1, 8)).to(BF).to(gpu)
    eg.engram_window_cache_fill(k, k, torch.tensor([-3, 1 << 40], device=gpu), torch.tensor([2], device=gpu), p.cache_k,
                                p.cache_v, sinks=2)
    torch.cuda.synchronize()
    assert torch.equal(p.cache_k[2, 0, :6], k[:, 0])


@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_what_has_left_the_window_is_gone(gpu, value):
    p = Pool(gpu, 2, 4, 2, 64, 16, 2, spare=3, seed=6)
    p.fill([25, 25], [0, 1])
    clean_k, clean_v = p.cache_k.clone(), p.cache_v.clone()
    j = 25 - 16  # the oldest token that the next row (position 25) does not see
    for cache in (p.cache_k, p.cache_v):
        cache[0, :, p.line(j)] = value
    p.step([0, 1])
    q = torch.ones((1, 4, 64), dtype=BF, device=gpu)
    o = torch.empty_like(q)
    ws = torch.empty(eg.engram_window_attn_step_workspace_bytes(1, 4, 2, 64, p.capacity), dtype=torch.uint8, device=gpu)
    clean_v[1, :, p.line(20)] = value
    eg.engram_window_attn_step(q, q[:, :2], q[:, :2], clean_k, clean_v, torch.tensor([1], device=gpu),
                               torch.tensor([25], device=gpu), o, ws, 16, sinks=2)
    assert not torch.isfinite(o).any()


@pytest.mark.parametrize("window", [100, 4000], ids=["one launch", "two launches"])
def test_captured_and_replayed(gpu, window):
    """A decode step in a graph, slots and positions changing between the replays."""
    b, hq, hk, d, sinks = 3, 10, 2, 128, 4
    p = Pool(gpu, 4, hq, hk, d, window, sinks, seed=7)
    p.fill([300, 1, 150], [0, 1, 2])
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((b, h, d), generator=g).to(BF).to(gpu) for h in (hq, hk, hk))
    slots, pos = torch.tensor([0, 1, 2], device=gpu), torch.tensor([300, 1, 150], device=gpu)
    need = eg.engram_window_attn_step_workspace_bytes(b, hq, hk, d, window + sinks)
    assert (need > 0) == (window == 4000)  # lists in parts, joined by a second launch

    def run(ck, cv, o, ws):
        eg.engram_window_attn_step(q, k, v, ck, cv, slots, pos, o, ws, window, sinks=sinks, scale=d ** -0.5)

    def buffers():
        return p.cache_k.clone(), p.cache_v.clone(), torch.empty_like(q), torch.empty(need, dtype=torch.uint8, device=gpu)
    want, kept = buffers(), buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*kept)
    for i in range(4):
        q.copy_(torch.randn(q.shape, generator=g).to(BF))
        slots.copy_(slots.flip(0))
        pos.copy_(pos.flip(0) + 1)
        graph.replay()
        run(*want)
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(want[:3], kept[:3]))
