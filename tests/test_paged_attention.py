"""Attention over a paged cache, in 16 and in 4 bits, against its definition in 64 bits; and a run of
append and attention as a program decodes with them."""

import ctypes
import math

import numpy as np
import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from paged_common import four_bits, places, sound_struct, tables
from prefix_common import prefix_check, prefix_sums
from window_common import window_plain

gpu = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
BR = "padding_causal_bottom_right"


class Case:
    """Queries behind `past` cached tokens. Every place of the cache that no query sees holds NaN, free pages and
    those before a window among them; rows of q that are no token hold 1e3."""

    def __init__(self, seed, lengths, past, page, hq, hkv, d, dtype, bits, window=0, sinks=0, slot=3, tail=2, spread=0.0):
        gen = torch.Generator().manual_seed(seed)
        self.__dict__.update(lengths=lengths, past=past, page=page, hq=hq, hkv=hkv, d=d, dtype=dtype, bits=bits, window=window,
                             sinks=sinks, scale=1 / math.sqrt(d))
        off = np.cumsum([0] + [(n + slot - 1) // slot * slot for n in lengths]).tolist()
        self.off, self.total = off, off[-1] + tail
        self.q = torch.full((self.total, hq, d), 1e3).to(dtype)
        wide = torch.exp(spread * torch.randn(d, generator=gen))
        for o, n in zip(off, lengths):
            self.q[o:o + n] = (torch.randn(n, hq, d, generator=gen) * wide).to(dtype)
        keys = [p + n if n else 0 for p, n in zip(past, lengths)]
        self.keys, self.offk = keys, np.cumsum([0] + keys).tolist()
        k, v = ((torch.randn(sum(keys), hkv, d, generator=gen) * w).to(dtype) for w in (wide, torch.ones(d)))
        self.table, self.pages = tables(keys, page, seed)
        rows, pages, slots = places(self.table, page, [0] * len(keys), keys, self.offk)
        live = torch.ones(len(rows), dtype=torch.bool)
        if window:  # positions that no query sees any more
            for b, (p, m) in enumerate(zip(past, keys)):
                for t in range(min(m, sinks), min(m, max(0, p + 1 - window))):
                    live[self.offk[b] + t] = False
            for b, (p, m) in enumerate(zip(past, keys)):  # and whole pages of them
                for n in range((m + page - 1) // page):
                    if not live[self.offk[b] + n * page:self.offk[b] + min(m, (n + 1) * page)].any():
                        self.table[b, n] = -3
        rows, pages, slots = rows[live], pages[live], slots[live]
        self.caches, self.kv = [], []
        for x in (k, v):
            if bits == 16:
                c = torch.full((self.pages, hkv, page, d), float("nan"), dtype=dtype)
                c[pages, :, slots] = x[rows]
                self.caches.append(c)
                self.kv.append(x)
            else:
                codes, meta, values = four_bits(x)
                c = torch.full((self.pages, hkv, page, d // 2), 0xA5, dtype=torch.uint8)
                m = torch.full((self.pages, hkv, page, d // 32, 2), float("nan"), dtype=dtype)
                c[pages, :, slots], m[pages, :, slots] = codes[rows], meta[rows]
                self.caches.append((c, m))
                self.kv.append(values)
        self.cu = [prefix_sums(lengths), torch.tensor(off, dtype=torch.int32)]

    def dev(self):
        if not hasattr(self, "on"):
            up = lambda c: tuple(t.cuda() for t in c) if self.bits == 4 else c.cuda()  # noqa: E731
            self.on = [self.q.cuda(), up(self.caches[0]), up(self.caches[1]), self.table.cuda(),
                       torch.tensor(self.past, dtype=torch.int32).cuda(), *(c.cuda() for c in self.cu)]
        return self

    def fwd(self, **kw):
        self.dev()
        return ta.paged_fwd(*self.on, self.scale, window=self.window, sinks=self.sinks, **kw)

    def workspace(self):
        n = ta.paged_fwd_workspace_size(len(self.lengths), self.total, self.hq, self.hkv, self.d, self.bits)
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def check(self):
        ws = self.workspace()
        out, lse = self.fwd(workspace=ws)
        assert ta.read_status(ws) == 0
        ref = window_plain(self.q, *self.kv, None, list(zip(self.off, self.lengths)), list(zip(self.offk, self.keys)), self.scale, BR,
                           self.window, self.sinks)
        prefix_check({"out": out, "lse": lse}, ref, ("out", "lse"), self.dtype)
        return out, lse


def _bits(ts):
    return [t.view(torch.int32 if t.dtype == torch.float32 else torch.int16).clone() for t in ts]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(_bits(a), _bits(b)))


# ------------------------------------------------------------------ on the CPU
def test_refusals():
    L, one, null = ta.library(), ctypes.c_void_p(4096), None

    def fwd(q=one, cu=one, past=one, batch=1, total=3, hq=2, scale=0.1, window=0, sinks=0, ws=one, size=0, **changes):
        c = sound_struct()
        for n, v in changes.items():
            setattr(c, n, v)
        return L.te_attn_paged_fwd_thd(ctypes.byref(c), q, one, one, cu, one, past, batch, total, hq, ctypes.c_float(scale), window, sinks, ws,
                                       ctypes.c_size_t(size), null)
    last = lambda: L.te_attn_last_error().decode()  # noqa: E731
    for kw, code, word in ((dict(q=null), -1, "NULL"), (dict(q=ctypes.c_void_p(4104)), -1, "aligned"), (dict(cu=null), -1, "cu_seqlens"),
                           (dict(past=ctypes.c_void_p(4098)), -1, "alignment"), (dict(batch=0), -1, "batch"), (dict(batch=4097), -2, "4096"),
                           (dict(total=-1), -1, "total_q"), (dict(hq=3), -1, "multiple"), (dict(scale=float("nan")), -1, "finite"),
                           (dict(window=-1), -1, "window"), (dict(window=4, sinks=-1), -1, "sinks"), (dict(sinks=4), -1, "sinks"), (dict(ws=null), -1, "NULL"),
                           (dict(), -3, "workspace"), (dict(page_size=12), -2, "page_size"), (dict(max_pages=1 << 27), -2, "2^30"),
                           (dict(total=2 ** 30, hq=2), -2, "large")):
        assert fwd(**kw) == code and word in last(), (kw, last())
    for bad in ((0, 4, 8, 2, 64, 16), (1, 4, 8, 3, 64, 16), (1, 4, 8, 2, 12, 16), (1, 4, 8, 2, 64, 8), (4097, 4, 8, 2, 64, 4)):
        assert ta.paged_fwd_workspace_size(*bad) == 0


def test_refusals_in_python():
    k, v = ta.paged_cache(4, 16, 2, 64, device="cpu")
    x, i, cu = torch.zeros(3, 2, 64, dtype=BF), torch.zeros(1, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ta.paged_fwd(x, k, v, i[None], i, cu, cu, 0.1)


# ------------------------------------------------------------------ on the GPU
CASES = [
    # lengths, past, page, hq, hkv, d, dtype, bits, window, sinks
    ([1, 1, 1], [0, 20, 199], 16, 8, 8, 64, FP, 16),
    ([1] * 9, [0, 15, 16, 17, 500, 3, 31, 32, 1200], 16, 8, 2, 128, BF, 16),
    ([1] * 9, [0, 15, 16, 17, 500, 3, 31, 32, 1200], 32, 8, 2, 128, BF, 4),
    ([1, 0, 4, 7, 2], [700, 30, 0, 90, 63], 64, 6, 2, 96, FP, 16),
    ([1, 0, 4, 7, 2], [700, 30, 0, 90, 63], 16, 6, 2, 96, FP, 4),
    ([50, 1, 130], [70, 900, 0], 16, 8, 2, 128, BF, 16),
    ([50, 1, 130], [70, 900, 0], 64, 8, 2, 128, FP, 4),
    ([3, 1], [2000, 1], 128, 16, 1, 256, BF, 16),
    ([3, 1], [2000, 1], 32, 16, 1, 256, FP, 4),
    ([1, 5, 1], [900, 600, 10], 16, 4, 2, 128, BF, 16, 100, 4),
    ([1, 5, 1], [900, 600, 10], 16, 4, 2, 128, BF, 4, 100, 4),
    ([1, 5, 20], [900, 600, 1000], 64, 4, 4, 64, FP, 16, 1, 0),
    ([1, 5, 20], [900, 600, 1000], 32, 4, 4, 64, FP, 4, 33, 0),
    ([40, 2], [300, 700], 32, 3, 1, 80, BF, 16, 64, 100),
    ([1, 3], [257, 40], 16, 2, 2, 8, FP, 16),
    ([1, 3], [257, 40], 16, 2, 2, 32, FP, 4),
    ([1, 3], [257, 40], 4096, 7, 1, 160, BF, 4),
    ([1, 3], [257, 40], 256, 24, 1, 192, FP, 16, 2 ** 31 - 1, 2 ** 31 - 1),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_against_the_definition(case):
    Case(41, *case).check()


@gpu
@pytest.mark.parametrize("seed", range(14))
def test_random(seed):
    r = np.random.default_rng(500 + seed)
    n = int(r.integers(1, 9))
    bits = [16, 4][seed % 2]
    hkv = int(r.integers(1, 4))
    lengths = [int(x) for x in (r.integers(0, 3, n) if seed % 3 else r.integers(0, 40, n))]
    past = [int(2 ** r.uniform(0, 10.5)) - 1 for _ in range(n)]
    window = int(r.choice([0, 0, int(2 ** r.uniform(0, 9))]))
    Case(seed, lengths, past, int(r.choice([16, 32, 64, 128])), hkv * int(r.integers(1, 10)), hkv,
         int(r.choice([32, 64, 96, 128, 224, 256])) if bits == 4 else 8 * int(r.integers(1, 33)), [BF, FP][int(r.integers(2))], bits, window,
         int(r.choice([0, 3, 50])) if window else 0, slot=int(r.integers(1, 4)), tail=int(r.integers(0, 3)), spread=0.5).check()


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_many_sequences_and_long_ones(bits):
    """More sequences than a block has threads, and few that each go over many warps."""
    Case(42, [1] * 500, [int(37 * i % 200) for i in range(500)], 16, 2, 1, 64, BF, bits, slot=1, tail=0).check()
    Case(43, [1, 2], [20000, 7], 64, 4, 2, 128, FP, bits, slot=1, tail=0).check()


WIDE = [
    # pieces of prompts: more than 64 rows a kv head go to the kernel of many rows
    ([200, 300], [0, 500], 16, 8, 2, 128, BF, 16),
    ([200, 300], [0, 500], 32, 8, 2, 128, BF, 4),
    ([129, 1, 64, 0, 700], [1000, 30, 5, 9, 0], 64, 4, 2, 64, FP, 16),
    ([129, 1, 64, 0, 700], [1000, 30, 5, 9, 0], 16, 4, 2, 64, FP, 4),
    ([90, 41], [400, 3000], 128, 3, 1, 96, BF, 16),             # groups that no tile holds whole
    ([90, 41], [400, 3000], 64, 10, 2, 96, BF, 4),
    ([30, 7], [700, 100], 256, 48, 1, 80, FP, 16),
    ([5, 3], [900, 100], 32, 300, 1, 64, BF, 16),               # more heads than a row tile
    ([300, 90], [900, 100], 16, 4, 1, 128, FP, 16, 100, 4),
    ([300, 90], [900, 100], 16, 4, 1, 128, FP, 4, 100, 4),
    ([300, 90], [900, 4000], 64, 4, 2, 64, BF, 16, 33, 0),
    ([300, 90], [900, 4000], 32, 4, 2, 64, BF, 4, 500, 300),
    ([140, 200], [2000, 30], 16, 6, 1, 256, BF, 16, 90, 2),     # (head_dim 256: the kernel of few rows takes them)
    ([140], [200], 16, 2, 1, 256, FP, 4),
    ([1500], [700], 64, 2, 1, 128, BF, 16),
]


@gpu
@pytest.mark.parametrize("case", WIDE, ids=[str(i) for i in range(len(WIDE))])
def test_pieces_of_prompts(case):
    Case(61, *case).check()


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_both_kernels_in_one_call(bits):
    """A piece of a prompt among decoding sequences gives what each gives alone, within what their
    tensors' type leaves, and repeats give the same bits."""
    c = Case(62, [1, 200, 1, 2, 1], [700, 300, 40, 5, 90], 16, 4, 2, 128, BF, bits)
    first = c.check()
    assert _same(first, c.fwd())
    with ta.debug_build():
        ws = c.workspace()
        assert _same(first, c.fwd(workspace=ws)) and ta.read_status(ws) == 0


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_pages_outside_the_cache_for_pieces(bits):
    """Their keys are seen by no query, and the call says so (the last token's keys alone differ)."""
    c = Case(63, [100], [300], 16, 2, 1, 64, FP, bits, slot=1, tail=0)
    table = c.table.clone()
    table[0, 3], table[0, 9] = -1, c.pages
    c.dev().on[3].copy_(table)
    ws = c.workspace()
    out, lse = c.fwd(workspace=ws)
    assert ta.read_status(ws) == 16
    # the same queries over a cache in which those pages hold keys that nothing sees: positions 48-63
    # and 144-159 lie before all queries, so leaving them out shifts no query's limit but by 32
    keep = torch.ones(400, dtype=torch.bool)
    keep[48:64] = keep[144:160] = False
    ref = window_plain(c.q, c.kv[0][keep], c.kv[1][keep], None, [(0, 100)], [(0, 368)], c.scale, BR, 0, 0)
    prefix_check({"out": out, "lse": lse}, ref, ("out", "lse"), FP)


@gpu
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("scale", [-0.9, 0.0])
def test_other_scales(bits, scale):
    """Negative ones, with scores far apart, and none at all, for both kernels."""
    c = Case(64, [1, 90], [300, 200], 16, 2, 1, 64, BF, bits)
    c.scale = scale
    c.check()


@gpu
def test_as_many_sequences_as_are_taken():
    Case(65, [1] * 4096, [i % 20 for i in range(4096)], 16, 1, 1, 8, FP, 16, slot=1, tail=0).check()


@gpu
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("growth", [4.0, -4.0])
def test_scores_that_climb(bits, growth):
    """Maxima that grow, or fall, by far more than 2^8 along the keys."""
    c = Case(44, [1, 3], [900, 400], 16, 4, 2, 64, BF, bits)
    u = torch.zeros(64)
    u[::4] = 1.0
    for b, m in enumerate(c.keys):
        step = torch.arange(m)[:, None, None] * growth / 16
        x = (c.kv[0][c.offk[b]:c.offk[b] + m].float() + step * u).to(BF)
        _, pages, slots = places(c.table[b:b + 1], 16, [0], [m], [0])
        if bits == 16:
            c.caches[0][pages, :, slots] = x
        else:
            codes, meta, x = four_bits(x)
            c.caches[0][0][pages, :, slots], c.caches[0][1][pages, :, slots] = codes, meta
        c.kv[0][c.offk[b]:c.offk[b] + m] = x
    c.q = torch.where(torch.arange(4)[:, None] % 2 == 0, c.q, (c.q.float() + u).to(BF))
    # (scores of hundreds: fp32's 2^-24 of them and of their products is far below 1e-3)
    out, lse = c.fwd()
    ref = window_plain(c.q, *c.kv, None, list(zip(c.off, c.lengths)), list(zip(c.offk, c.keys)), c.scale, BR, 0, 0)
    prefix_check({"out": out, "lse": lse}, ref, ("out", "lse"), BF, lse_tol=1e-3)


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_repeats_and_what_buffers_held(bits):
    c = Case(45, [1, 0, 2, 30], [700, 5, 33, 64], 32, 4, 2, 128, BF, bits)
    first = c.fwd()
    poison = lambda t: torch.full_like(t.view(torch.uint8), 255).view(t.dtype)  # noqa: E731
    ws = c.workspace()
    assert _same(first, c.fwd(out=poison(first[0]), lse=poison(first[1]), workspace=ws))
    other = Case(46, [3, 1, 2, 29], [70, 500, 3, 6], 32, 4, 2, 128, BF, bits)  # a workspace that another call left
    other.fwd(workspace=ws)
    assert _same(first, c.fwd(workspace=ws)) and ta.read_status(ws) == 0


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_debug_build_finds_nothing(bits):
    c = Case(47, [1, 40, 2], [700, 5, 33], 16, 6, 2, 96, FP, bits, 50, 3)
    first = c.fwd()
    with ta.debug_build():
        ws = c.workspace()
        assert _same(first, c.fwd(workspace=ws)) and ta.read_status(ws) == 0


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_pages_outside_the_cache(bits):
    """Their keys are not seen, and the call says so; without any key the row is empty."""
    c = Case(48, [1, 1, 1], [99, 40, 10], 16, 2, 1, 64, FP, bits, slot=1, tail=0)
    for page in (-1, c.pages, 2 ** 31 - 1):
        table = c.table.clone()
        table[0, 2], table[2, 0] = page, page
        c.dev().on[3].copy_(table)
        ws = c.workspace()
        out, lse = c.fwd(workspace=ws)
        assert ta.read_status(ws) == 16
        keep = torch.ones(sum(c.keys), dtype=torch.bool)
        keep[32:48] = False
        ref = window_plain(c.q, c.kv[0][keep], c.kv[1][keep], None, [(0, 1), (1, 1), (2, 1)], [(0, 84), (84, 41), (125, 0)], c.scale, BR, 0, 0)
        prefix_check({"out": out, "lse": lse}, ref, ("out", "lse"), FP)
        assert lse[2].isneginf().all() and not out[2].any()


@gpu
def test_lengths_that_do_not_fit():
    """A past that is negative or runs past the page table, and lengths past their slots: empty, and reported."""
    c = Case(49, [2, 1, 3], [60, 20, 5], 16, 2, 1, 64, BF, 16, slot=4, tail=0).dev()
    whole = c.fwd()[0]
    for where, value in ((4, [-1, 20, 5]), (4, [60, 20000, 5]), (4, [60, 2 ** 31 - 1, 5]), (5, [0, 2, 12, 15])):
        kept = c.on[where].clone()
        c.on[where].copy_(torch.tensor(value, dtype=torch.int32))
        ws = c.workspace()
        out, lse = c.fwd(workspace=ws)
        assert ta.read_status(ws) == 1
        bad = 0 if value[0] == -1 else 1
        for b in range(3):
            rows = slice(c.off[b], c.off[b] + 4)
            assert torch.equal(out[rows], torch.zeros_like(out[rows]) if b == bad else whole[rows]), (value, b)
        c.on[where].copy_(kept)


@gpu
def test_nothing_to_do():
    c = Case(50, [0, 0], [10, 0], 16, 2, 1, 64, BF, 16, tail=3)
    ws = c.workspace()
    out, lse = c.fwd(workspace=ws)
    assert not out.any() and not lse.any() and ta.read_status(ws) == 0
    e = ta.paged_fwd(c.on[0][:0], *c.on[1:5], torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), 0.1,
                     workspace=ws)
    assert e[0].shape == (0, 2, 64) and ta.read_status(ws) == 0


@gpu
def test_a_nan_that_a_row_sees_is_passed_on():
    c = Case(51, [1, 1], [100, 100], 16, 2, 1, 64, BF, 16, slot=1, tail=0)
    p = int(c.table[0, 3])
    c.caches[1][p, 0, 5, 7] = float("nan")
    out, lse = c.fwd()
    assert torch.isnan(out[0, :, 7]).all() and torch.isfinite(out[0, :, :7]).all() and torch.isfinite(out[1]).all() and torch.isfinite(lse).all()


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_decoding_in_a_graph(bits):
    """Eight steps of append and attention, captured once and replayed with past counted up, against
    attention over everything at once: a prompt's tokens and the steps' in one packed batch."""
    hq, hkv, d, page, B, steps = 4, 2, 64, 16, 3, 8
    prompt = [5, 40, 17]
    gen = torch.Generator().manual_seed(52)
    rnd = lambda n, h: torch.randn(n, h, d, generator=gen).to(BF).cuda()  # noqa: E731
    total = [n + steps for n in prompt]
    q, k, v = rnd(sum(total), hq), rnd(sum(total), hkv), rnd(sum(total), hkv)
    off = np.cumsum([0] + total).tolist()
    w, _ = ta.rope_frequencies(d)
    table, pages = tables(total, page, 3)
    table = table.cuda()
    caches = ta.paged_cache(pages, page, hkv, d, BF, bits)
    window = dict(window=24, sinks=2)
    past = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = torch.cat([torch.arange(o, o + n) for o, n in zip(off, prompt)]).cuda()
    cu = prefix_sums(prompt).cuda()
    got = torch.zeros(sum(total), hq, d, dtype=BF, device="cuda")
    lse = torch.zeros(sum(total), hq, device="cuda")

    def step(x, cu):
        turned = ta.paged_append(*x, *caches, table, past, cu, cu, inv_freq=w)
        return ta.paged_fwd(turned, *caches, table, past, cu, cu, 0.125, **window)
    got[rows], lse[rows] = step([t[rows] for t in (q, k, v)], cu)
    past += torch.tensor(prompt, dtype=torch.int32, device="cuda")
    one = prefix_sums([1] * B).cuda()
    buf = [torch.zeros(B, h, d, dtype=BF, device="cuda") for h in (hq, hkv, hkv)]
    ends = torch.tensor([o + n for o, n in zip(off, prompt)]).cuda()
    spare = past.clone()
    step(buf, one)  # (the entry points' first calls come before a capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(buf, one)
        past += 1
    past.copy_(spare)
    for s in range(steps):
        for b, t in zip(buf, (q, k, v)):
            b.copy_(t[ends + s])
        graph.replay()
        got[ends + s], lse[ends + s] = out
    cu = prefix_sums(total).cuda()
    qr, kr = ta.rope(q, k, w, cu, cu)
    if bits == 4:
        kr, v = (four_bits(t)[2].cuda() for t in (kr, v))
    spans = list(zip(off, total))
    ref = window_plain(qr, kr, v, None, spans, spans, 0.125, BR, 24, 2)
    prefix_check({"out": got, "lse": lse}, ref, ("out", "lse"), BF)
    # and what a model trained with that window computes
    if bits == 16:
        same = ta.window_fwd(qr, kr, v, cu, cu, cu, cu, 0.125, 24, 2)
        prefix_check({"out": same[0], "lse": same[1]}, ref, ("out", "lse"), BF)


@gpu
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("window", [0, 100])
def test_prompts_of_many_row_tiles(bits, window):
    """More row tiles than a warp looks through at once, in sequences on both sides of one of few rows."""
    Case(66, [700, 1, 560], [40, 90, 0], 64, 17, 1, 64, BF, bits, window, 3 if window else 0).check()


@gpu
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("n", [1, 60])
def test_pages_that_sequences_share(bits, n):
    """Two sequences over the same pages, the same page twice in one of them, and a table whose rows are
    slices of wider ones, against a cache in which every sequence has copies of its own."""
    c = Case(67, [n] * 2, [64 * 5 - n] * 2, 64, 8, 2, 128, BF, bits, slot=1, tail=0).dev()
    table = torch.full((2, 40), -9, dtype=torch.int32, device="cuda")
    table[0, 3:8] = c.on[3][0, :5]
    table[1, 3:8] = c.on[3][0, :5]
    table[1, 5] = table[1, 3]
    shared = ta.paged_fwd(*c.on[:3], table[:, 3:8], *c.on[4:], c.scale)
    own = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
    pages = table[:, 3:8].flatten().long()
    copies = [tuple(t[pages].clone() for t in x) if bits == 4 else x[pages].clone() for x in c.on[1:3]]
    assert _same(shared, ta.paged_fwd(c.on[0], *copies, own, *c.on[4:], c.scale))


@gpu
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("n", [1, 60])
def test_offsets_past_32_bits(bits, n):
    """Pages that begin more than 4 GiB, and 2^31 elements, into the cache."""
    c = Case(68, [n, 1], [300, 5], 64, 32, 8, 128, BF, bits).dev()
    first = c.fwd()
    far = 40000 * (4 if bits == 4 else 1)
    large = ta.paged_cache(far + c.pages, 64, 8, 128, BF, bits)
    for big, x in zip(large, c.on[1:3]):
        for a, b in zip(big, x) if bits == 4 else ((big, x),):
            a[far:].copy_(b)
    table = torch.where(c.on[3] >= 0, c.on[3] + far, c.on[3])
    assert _same(first, ta.paged_fwd(c.on[0], *large, table, *c.on[4:], c.scale))


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_two_streams_at_once(bits):
    """Calls in flight on two streams, each with its own workspace, do not touch each other."""
    cs = [Case(s, [1] * 20 + [90, 130], [(s + 41 * i) % 700 for i in range(20)] + [500, 30], 32, 8, 2, 128, BF, bits).dev() for s in (69, 70)]
    refs = [[x.clone() for x in c.fwd()] for c in cs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, (c, st) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(st):
                got[i].append(c.fwd())
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert _same(refs[i], g)


@gpu
def test_given_outputs_and_streams():
    c = Case(71, [1, 90, 3], [300, 20, 64], 16, 4, 2, 64, BF, 16).dev()
    want = c.fwd()
    o, l = torch.full_like(want[0], float("nan")), torch.full_like(want[1], float("nan"))
    got = c.fwd(out=o, lse=l)
    assert got[0] is o and got[1] is l and _same(want, got)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        a = c.fwd(stream=side.cuda_stream)
        torch.empty(1 << 20, device="cuda").fill_(float("nan"))  # of the current stream's memory
        side.synchronize()
        assert _same(want, a)
    assert not any(x.requires_grad for x in ta.paged_fwd(c.on[0].clone().requires_grad_(), *c.on[1:], c.scale))
    for bad in (dict(out=o[:-1]), dict(lse=l.double()), dict(out=o.half()), dict(lse=l[:, :1])):
        with pytest.raises(ValueError):
            c.fwd(**bad)
    with pytest.raises(ta.TeAttnError, match="workspace"):
        c.fwd(workspace=c.workspace()[:-256])
    assert _same(want, c.fwd())


@gpu
def test_captured_calls_that_share_a_workspace():
    """Two captured calls of different shapes, one workspace, replayed in turn on one stream."""
    a, b = (Case(s, n, p, 16, 4, 2, 128, BF, 16).dev() for s, n, p in ((72, [1, 70], [400, 60], ), (73, [90, 2, 1], [30, 0, 800])))
    want = [a.fwd(), b.fwd()]
    ws = max((c.workspace() for c in (a, b)), key=lambda t: t.numel())
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph, c in zip(graphs, (a, b)):
        with torch.cuda.graph(graph):
            outs.append(c.fwd(workspace=ws))
    for _ in range(3):
        for i in range(2):
            outs[i][0].fill_(float("nan"))
            graphs[i].replay()
            torch.cuda.synchronize()
            assert _same(want[i], outs[i]) and ta.read_status(ws) == 0


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_prompts_among_many_sequences(bits):
    """So many sequences that one block of the join takes all heads of one; drafts, whose queries several share; rows
    between them that are no token."""
    Case(74, [1] * 1300 + [70], [7 * i % 90 for i in range(1300)] + [20], 16, 32, 2, 32, BF, bits).check()
    Case(75, [4, 3, 0, 64, 2], [3000, 700, 9, 40, 1200], 32, 8, 8, 64, FP, bits, tail=40).check()


@gpu
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("d", [64, 128])
def test_drafts_of_many_sequences(d, bits):
    """With segments for every SM, sequences of 16, or 32, rows go to the tensor cores and those of fewer do not."""
    Case(76, [5, 3, 9, 20, 0, 4, 8] * 24, [13 * i % 400 for i in range(168)], 32, 4, 1, d, FP, bits, slot=1).check()
    Case(77, [5, 3, 9, 20, 0, 4, 8] * 24, [13 * i % 400 for i in range(168)], 16, 4, 1, d, BF, bits, 60, 2, slot=1).check()


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_lengths_that_do_not_fit_among_prompts(bits):
    """The same where the kernel of many rows is launched: rows of such a sequence are zeros, the others' are theirs."""
    c = Case(78, [300, 2, 150], [60, 20, 5], 16, 4, 2, 64, BF, bits, slot=4, tail=3).dev()
    whole = c.fwd()
    for value in ([-1, 20, 5], [60, 20000, 5], [60, 20, 2 ** 31 - 1]):
        kept = c.on[4].clone()
        c.on[4].copy_(torch.tensor(value, dtype=torch.int32))
        ws = c.workspace()
        out, lse = c.fwd(workspace=ws)
        assert ta.read_status(ws) == 1
        for b in range(3):
            rows = slice(c.off[b], c.off[b + 1])
            good = value[b] == c.past[b]
            assert torch.equal(out[rows], whole[0][rows] if good else torch.zeros_like(out[rows])), (value, b)
            assert torch.equal(lse[rows], whole[1][rows] if good else torch.zeros_like(lse[rows])), (value, b)
        assert not out[c.off[3]:].any() and not lse[c.off[3]:].any()
        c.on[4].copy_(kept)
