"""Appending to a paged cache and reading it back, in 16 and in 4 bits."""

import ctypes

import numpy as np
import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from paged_common import CacheStruct, four_bits, places, sound_struct, tables
from prefix_common import prefix_sums, rope_check, rope_plain

gpu = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


class Case:
    """New tokens of packed sequences behind `past` ones; the cache holds the bytes 0x5a before."""

    def __init__(self, seed, lengths, past, page, hq, hkv, d, dtype, bits, rot, interleaved=False, fused=True, slot=3, tail=2,
                 shift=0):
        gen = torch.Generator().manual_seed(seed)
        self.__dict__.update(lengths=lengths, past=past, page=page, hq=hq, hkv=hkv, d=d, dtype=dtype, bits=bits, rot=rot,
                             interleaved=interleaved)
        off = np.cumsum([0] + [(n + slot - 1) // slot * slot for n in lengths]).tolist()
        self.off, self.total = off, off[-1] + tail
        heads = hq + 2 * hkv
        flat = torch.randn(self.total * heads * d + shift, generator=gen).to(dtype)
        x = flat[shift:].view(self.total, heads, d)  # (with a shift, off every wide alignment)
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        if not fused:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.table, self.pages = tables([p + n for p, n in zip(past, lengths)], page, seed)
        self.w = ta.rope_frequencies(rot, device="cpu")[0] if rot else None
        self.cu = [prefix_sums(lengths), torch.tensor(off, dtype=torch.int32)]
        self.shift = shift

    def fresh(self):
        caches = ta.paged_cache(self.pages, self.page, self.hkv, self.d, self.dtype, self.bits)
        for c in caches:
            for t in (c if self.bits == 4 else (c,)):
                t.view(torch.uint8).fill_(0x5A)
        return caches

    def dev(self):
        if not hasattr(self, "on"):
            # one allocation, so that strides and alignment stay
            base = self.q._base if self.q._base is not None else None
            if base is not None and base is self.k._base:
                flat = base.cuda()
                view = lambda t: flat.as_strided(t.shape, t.stride(), t.storage_offset())  # noqa: E731
                self.on = [view(t) for t in (self.q, self.k, self.v)]
            else:
                self.on = [t.cuda() for t in (self.q, self.k, self.v)]
            self.table_on, self.past_on = self.table.cuda(), torch.tensor(self.past, dtype=torch.int32).cuda()
            self.cu_on = [c.cuda() for c in self.cu]
            self.w_on = None if self.w is None else self.w.cuda()
        return self

    def append(self, caches, with_q=True, **kw):
        self.dev()
        q, k, v = self.on
        return ta.paged_append(q if with_q else None, k, v, *caches, self.table_on, self.past_on, *self.cu_on, inv_freq=self.w_on,
                               interleaved=self.interleaved, **kw)

    def gather(self, caches, **kw):
        self.dev()
        return ta.paged_gather(*caches, self.table_on, self.past_on, *self.cu_on, self.total, **kw)

    def check(self):
        caches, status = self.fresh(), torch.full((1,), 77, dtype=torch.int32, device="cuda")
        q = self.append(caches, status=status)
        assert status.item() == 0
        turned = [self.q, self.k]
        if self.rot:  # what the rotation alone gives, to the bit, and near the definition
            self.dev()
            turned = [t.cpu() for t in ta.rope(self.on[0], self.on[1], self.w_on, *self.cu_on, start_positions=self.past_on,
                                               interleaved=self.interleaved)]
            for got, x in ((q, self.q), (turned[1], self.k)):
                ref, size = rope_plain(x, self.w, self.lengths, self.off, self.past, self.interleaved, 1.0)
                rope_check(got, ref, size)
        rows, pages, slots = places(self.table, self.page, self.past, self.lengths, self.off)
        real = torch.zeros(self.total, dtype=torch.bool)
        real[rows] = True
        q = q.cpu()
        assert torch.equal(q[real], turned[0][real]) and not q[~real].any()
        got = self.gather(caches, status=status)
        assert status.item() == 0
        for kv, (cache, x) in enumerate(zip(caches, (turned[1], self.v))):
            parts = cache if self.bits == 4 else (cache,)
            want = list(self.fresh()[kv]) if self.bits == 4 else [self.fresh()[kv]]
            want = [t.cpu() for t in want]
            values = x
            if self.bits == 4:
                codes, meta, values = four_bits(x)
                want[0][pages, :, slots], want[1][pages, :, slots] = codes[rows], meta[rows]
            else:
                want[0][pages, :, slots] = x[rows]
            for a, b in zip(parts, want):  # new places as defined, all others as they were
                assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
            held = torch.zeros(self.total, self.hkv, self.d, dtype=self.dtype)
            held[rows] = values[rows]
            assert torch.equal(got[kv].cpu(), held)


# ------------------------------------------------------------------ on the CPU
def test_four_bits_by_hand():
    x = torch.arange(32, dtype=torch.float32)[None]  # least 0, step 31 / 15 = 2.0666 -> bf16 2.0625
    codes, meta, value = four_bits(x.to(BF))
    assert meta.tolist() == [[[2.0625, 0.0]]]
    assert codes[0, 0].item() == 0 and codes[0, 1].item() == (1 | 1 << 4)  # 0, 0.48 -> 0, 0; 0.97, 1.45 -> 1, 1
    assert codes[0, 15].item() == (15 | 15 << 4) and value[0, 31].item() == 31.0  # 30.9375 in bf16
    same, _, value = four_bits(torch.full((1, 32), 3.5, dtype=FP))
    assert not same.any() and (value == 3.5).all()


def _last():
    return ta.library().te_attn_last_error().decode()


@pytest.mark.parametrize("bits", [16, 4])
def test_refusals_of_a_cache(bits):
    L, one, null = ta.library(), ctypes.c_void_p(4096), None

    def gather(**changes):
        c = sound_struct(bits)
        for n, v in changes.items():
            setattr(c, n, v)
        return L.te_attn_paged_gather(ctypes.byref(c), one, one, one, one, one, 1, 0, null, null)
    assert gather() == 0  # no rows: nothing is launched
    for changes, code, word in (({"page_size": 8}, -2, "page_size"), ({"page_size": 24}, -2, "page_size"), ({"page_size": 8192}, -2, "page_size"),
                                ({"d": 12}, -2, "head dim"), ({"d": 264}, -2, "head dim"), ({"hkv": 0}, -1, "hkv"), ({"hkv": 5000}, -2, "heads"),
                                ({"num_pages": 0}, -1, "num_pages"), ({"max_pages": 0}, -1, "max_pages"), ({"dtype": 3}, -2, "dtype"),
                                ({"k": 4100}, -1, "aligned"), ({"v": 0}, -1, "NULL"), ({"page_table": 0}, -1, "NULL"),
                                ({"page_table": 4098}, -1, "alignment"), ({"k_stride": 64}, -1, "strides"), ({"v_stride": 1 << 62}, -1, "strides"),
                                ({"k_stride": 65536 + 8}, -1, "strides"), ({"table_stride": -1}, -1, "table_stride"),
                                ({"v_meta": 0 if bits == 4 else 4096}, -1, "together")):
        assert gather(**changes) == code and word in _last(), (changes, _last())
    if bits == 4:
        assert gather(d=40) == -2 and "multiple of 32" in _last()
        assert gather(k_meta_stride=16) == -1 and "strides" in _last()
    assert L.te_attn_paged_gather(null, one, one, one, one, one, 1, 0, null, null) == -1 and "cache" in _last()


def test_refusals_of_an_append():
    L, one, null = ta.library(), ctypes.c_void_p(4096), None
    i64 = ctypes.c_int64

    def append(q=one, k=one, v=one, qo=one, w=one, n_freq=8, cu=one, past=one, batch=1, total=3, hq=2, stride=128, mscale=1.0, status=null):
        return L.te_attn_paged_append(ctypes.byref(sound_struct()), q, k, v, qo, w, n_freq, cu, one, past, batch, total, hq,
                                      *[i64(stride)] * 6, 0, ctypes.c_float(mscale), status, null)
    for kw, code, word in ((dict(k=null), -1, "NULL"), (dict(qo=null), -1, "NULL"), (dict(w=null), -1, "inv_freq"), (dict(n_freq=33), -1, "n_freq"),
                           (dict(n_freq=-1), -1, "n_freq"), (dict(cu=null), -1, "cu_seqlens"), (dict(past=null), -1, "positions"),
                           (dict(batch=0), -1, "batch"), (dict(total=-1), -1, "rows"), (dict(total=2 ** 31 - 1), -1, "rows"), (dict(hq=-1), -1, "hq"),
                           (dict(hq=5000), -2, "heads"), (dict(stride=-1), -1, "strides"), (dict(stride=2 ** 31 + 1), -1, "strides"),
                           (dict(mscale=float("inf")), -1, "mscale"), (dict(k=ctypes.c_void_p(4097)), -1, "aligned"),
                           (dict(w=ctypes.c_void_p(4100)), -1, "alignment"), (dict(past=ctypes.c_void_p(4098)), -1, "alignment"),
                           (dict(status=ctypes.c_void_p(4098)), -1, "alignment")):
        assert append(**kw) == code and word in _last(), (kw, _last())
    assert ctypes.sizeof(CacheStruct) == 104


def test_refusals_in_python():
    k, v = ta.paged_cache(4, 16, 2, 64, device="cpu")
    x, i = torch.zeros(3, 2, 64, dtype=BF), torch.zeros(1, dtype=torch.int32)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ta.paged_append(x, x, x, k, v, i[None], i, cu, cu)
    with pytest.raises(ValueError, match="CUDA"):
        ta.paged_gather(k, v, i[None], i, cu, cu, 3)
    for bad in (dict(bits=8), dict(bits=4, d=40), dict(dtype=torch.float32)):
        with pytest.raises(ValueError):
            ta.paged_cache(4, 16, 2, **{"d": 64, "device": "cpu", **bad})


# ------------------------------------------------------------------ on the GPU
CASES = [
    # lengths, past, page, hq, hkv, d, dtype, bits, rot, interleaved, fused, ...
    dict(lengths=[1] * 7, past=[0, 15, 16, 17, 900, 3, 31], page=16, hq=8, hkv=2, d=128, dtype=BF, bits=16, rot=128, slot=1, tail=0),
    dict(lengths=[1] * 7, past=[0, 15, 16, 17, 900, 3, 31], page=16, hq=8, hkv=2, d=128, dtype=BF, bits=4, rot=128, slot=1, tail=0),
    dict(lengths=[40, 0, 1, 33], past=[0, 5, 130000, 63], page=64, hq=3, hkv=1, d=64, dtype=FP, bits=16, rot=32, interleaved=True),
    dict(lengths=[40, 0, 1, 33], past=[0, 5, 1300, 63], page=32, hq=3, hkv=1, d=64, dtype=FP, bits=4, rot=32, interleaved=True),
    dict(lengths=[5, 9], past=[2, 0], page=16, hq=2, hkv=2, d=80, dtype=BF, bits=16, rot=40, fused=False),
    dict(lengths=[5, 9], past=[2, 0], page=16, hq=2, hkv=2, d=96, dtype=BF, bits=4, rot=24, fused=False),
    dict(lengths=[17, 3], past=[2, 0], page=128, hq=5, hkv=1, d=256, dtype=FP, bits=4, rot=64, shift=1),
    dict(lengths=[17, 3], past=[2, 0], page=128, hq=5, hkv=1, d=256, dtype=FP, bits=16, rot=64, shift=1),
    dict(lengths=[17, 3], past=[2, 0], page=16, hq=2, hkv=2, d=32, dtype=BF, bits=4, rot=32, shift=2, interleaved=True),
    dict(lengths=[17, 3], past=[2, 0], page=16, hq=2, hkv=2, d=32, dtype=BF, bits=4, rot=30, shift=4, interleaved=True),
    dict(lengths=[700, 2000, 1], past=[2, 0, 4000], page=32, hq=8, hkv=8, d=128, dtype=BF, bits=16, rot=128),
    dict(lengths=[700, 2000, 1], past=[2, 0, 4000], page=32, hq=4, hkv=8, d=128, dtype=FP, bits=4, rot=64),
    dict(lengths=[3, 2], past=[1, 30], page=16, hq=1, hkv=1, d=8, dtype=FP, bits=16, rot=2),
    dict(lengths=[3, 2], past=[1, 30], page=16, hq=1, hkv=1, d=64, dtype=FP, bits=4, rot=0),
    dict(lengths=[3, 2], past=[1, 30], page=16, hq=70, hkv=40, d=192, dtype=BF, bits=4, rot=192),
    dict(lengths=[3, 2], past=[1, 30], page=4096, hq=2, hkv=2, d=64, dtype=BF, bits=16, rot=0),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_append_and_gather(case):
    Case(31, **case).check()


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_caches_side_by_side(bits):
    """Keys and values of one tensor, a layer of several, and rows of a longer page table."""
    c = Case(32, [5, 1, 18], [3, 60, 14], 16, 4, 2, 64, BF, bits, 64).dev()
    plain = c.fresh()
    q = c.append(plain)
    lead = (c.pages, 3, 2, 2, 16)  # layers, keys and values
    if bits == 16:
        big = torch.zeros(*lead, 64, dtype=BF, device="cuda")
        caches = (big[:, 1, 0], big[:, 1, 1])
    else:
        codes, meta = torch.zeros(*lead, 32, dtype=torch.uint8, device="cuda"), torch.zeros(*lead, 2, 2, dtype=BF, device="cuda")
        caches = tuple((codes[:, 1, i], meta[:, 1, i]) for i in range(2))
    table = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
    table[:, 8:8 + c.table.shape[1]] = c.table_on
    c.table_on = table[:, 8:8 + c.table.shape[1]]
    assert torch.equal(q, c.append(caches))
    want = c.gather(plain)
    assert all(torch.equal(a, b) for a, b in zip(c.gather(caches), want))
    if bits == 16:
        assert not big[:, 0].any() and not big[:, 2].any()
    else:
        assert not any(t[:, i].any() for t in (codes, meta) for i in (0, 2))


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_pages_outside_the_cache(bits):
    """Tokens whose page is out of range, or behind the table, are reported and not written; the
    others are, and lengths that do not fit leave their sequence out."""
    c = Case(33, [20, 6, 40], [0, 10, 0], 16, 2, 1, 64, FP, bits, 64).dev()
    sound = c.fresh()
    q = c.append(sound)
    whole = c.gather(sound)
    for b, n, page in ((0, 1, c.pages), (1, 0, -1), (2, 2, 2 ** 31 - 1)):
        t = c.table.clone()
        t[b, n] = page
        c.table_on = t.cuda()
        caches, status = c.fresh(), torch.zeros(1, dtype=torch.int32, device="cuda")
        assert torch.equal(q, c.append(caches, status=status)) and status.item() == 16
        got = c.gather(caches, status=status)
        assert status.item() == 16
        lost = [c.off[b] + i for i in range(c.lengths[b]) if (c.past[b] + i) // 16 == n]
        for x, y in zip(got, whole):
            y = y.clone()
            y[lost] = 0
            assert torch.equal(x, y)
    c.table_on = c.table[:, :2].contiguous().cuda()  # the third sequence's last page is behind it
    caches = c.fresh()
    c.append(caches, status=status)
    assert status.item() == 16
    c.table_on = c.table.cuda()
    for name, change in (("past", lambda: c.past_on.__setitem__(1, -3)), ("len", lambda: c.cu_on[0].copy_(torch.tensor([0, 22, 26, 66])))):
        caches = c.fresh()
        kept = [t.clone() for t in (c.past_on, c.cu_on[0])]
        change()
        out = c.append(caches, status=status)
        assert status.item() == 1, name
        seq = 1 if name == "past" else 0
        assert not out[c.off[seq]:c.off[seq + 1]].any()
        c.past_on.copy_(kept[0])
        c.cu_on[0].copy_(kept[1])


@gpu
@pytest.mark.parametrize("dtype", [BF, FP])
def test_numbers_that_are_hard_to_hold(dtype):
    """The type's greatest and least, a group without a range, tiny ones, NaN and infinities."""
    big = torch.finfo(dtype).max
    c = Case(34, [9], [0], 16, 1, 1, 32, dtype, 4, 0, fused=False, tail=0, slot=1)
    v = torch.randn(9, 1, 32)
    v[0] = torch.where(v[0] > 0, big, -big)
    v[1], v[2] = big, 0
    v[3] *= float(torch.finfo(dtype).tiny)
    v[4, 0, 5], v[5, 0, 31], v[6, 0, 0] = float("nan"), float("inf"), -float("inf")
    v[7, 0, 3] = big
    c.v = v.to(dtype)
    caches = c.fresh()
    c.append(caches, with_q=False)
    got = c.gather(caches)[1].cpu()
    want = four_bits(c.v)[2]
    # (rounding twice in the plain form may move a tie: half a step of the type, 2^-9 or 2^-12, of each)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)) and torch.isnan(got[4:7]).all()
    err = (got.double() - want.double()).abs()[fine]
    assert (err <= torch.finfo(dtype).eps * want.double().abs()[fine] + 2 * torch.finfo(dtype).tiny * torch.finfo(dtype).eps).all()


@gpu
def test_without_queries_and_given_outputs():
    c = Case(35, [4, 2], [1, 20], 16, 2, 2, 64, BF, 16, 64).dev()
    a, b = c.fresh(), c.fresh()
    assert c.append(a, with_q=False) is None
    out = torch.empty(c.total, 2, 64, dtype=BF, device="cuda")
    assert c.append(b, q_out=out) is out
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    k, v = (torch.empty(c.total, 2, 64, dtype=BF, device="cuda") for _ in range(2))
    got = c.gather(a, k=k, v=v)
    assert got[0] is k and got[1] is v
    for bad in (dict(q_out=out[:-1]), dict(status=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            c.append(b, **bad)
    with pytest.raises(ValueError):
        c.append((b[0], b[1].half()))
    with pytest.raises(ValueError):
        c.append((b[0].transpose(1, 2), b[1].transpose(1, 2)))


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_graph_and_streams(bits):
    """A captured append follows past, tables and inputs; another stream gives the same."""
    c = Case(36, [1, 1, 1], [4, 15, 40], 16, 2, 1, 64, BF, bits, 64, slot=1, tail=0).dev()
    want, caches = c.fresh(), c.fresh()
    c.append(caches)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = c.append(caches)
    for step in range(3):
        c.past_on += 1
        c.on[1].copy_(torch.randn(3, 1, 64, generator=torch.Generator().manual_seed(step)))
        c.table_on.copy_(torch.where(c.table < 0, 0, c.table))
        graph.replay()
        ref = c.append(want)
        assert torch.equal(q, ref)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = c.append(want, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(other, ref)


def test_tables_of_too_many_pages_are_refused():
    """Positions stay below 2^30 for every call on a cache."""
    L, one, null = ta.library(), ctypes.c_void_p(4096), None
    for pages, page, code in ((2 ** 26, 16, 0), (2 ** 26 + 1, 16, -2), (2 ** 31 - 1, 16, -2), (2 ** 18, 4096, 0), (2 ** 18 + 1, 4096, -2)):
        c = sound_struct(page=page)
        c.max_pages = pages
        assert L.te_attn_paged_gather(ctypes.byref(c), one, one, one, one, one, 1, 0, null, null) == code, (pages, page)
        assert L.te_attn_paged_append(ctypes.byref(c), null, null, null, null, null, 0, one, one, one, 1, 0, 0, *[ctypes.c_int64(0)] * 6, 0,
                                      ctypes.c_float(1.0), null, null) == code, (pages, page)
        if code:
            assert "2^30" in _last()


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_offsets_past_32_bits(bits):
    """Pages whose bytes begin more than 4 GiB, and whose elements more than 2^31, into the cache."""
    c = Case(37, [70, 1], [30, 200], 64, 4, 8, 128, BF, bits, 64).dev()
    small, far = c.fresh(), 40000 * (4 if bits == 4 else 1)
    large = ta.paged_cache(far + c.pages, 64, 8, 128, BF, bits)
    q = c.append(small)
    first = c.gather(small)
    c.table_on = torch.where(c.table_on >= 0, c.table_on + far, c.table_on)
    assert torch.equal(q, c.append(large))
    assert all(torch.equal(a, b) for a, b in zip(first, c.gather(large)))


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_queries_turned_in_place(bits):
    c = Case(38, [40, 3], [0, 20], 16, 3, 1, 96, FP, bits, 64, fused=False).dev()
    a, b = c.fresh(), c.fresh()
    want = c.append(a)
    got = c.append(b, q_out=c.on[0])
    assert got is c.on[0] and torch.equal(want, got)


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_two_appends_at_once(bits):
    """On two streams, into caches of their own."""
    cs = [Case(s, [300, 1, 70], [5, 90, 0], 32, 8, 2, 128, BF, bits, 128).dev() for s in (39, 40)]
    want = [c.fresh() for c in cs]
    qs = [c.append(w) for c, w in zip(cs, want)]
    refs = [c.gather(w) for c, w in zip(cs, want)]
    fresh, streams = [c.fresh() for c in cs], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append((cs[i].append(fresh[i]), *cs[i].gather(fresh[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(x, y) for x, y in zip((qs[i], *refs[i]), g))


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_pages_read_by_several(bits):
    """Sequences that share the pages of a common beginning, out of a table with rows wider than it."""
    c = Case(41, [100, 20], [0, 90], 16, 2, 2, 64, BF, bits, 0).dev()
    caches = c.fresh()
    c.append(caches)
    wide = torch.full((4, 20), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[0, :7], wide[3, :7] = c.table_on[0, :7], c.table_on[0, :7]
    cu = torch.tensor([0, 100, 200], dtype=torch.int32, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    k, v = ta.paged_gather(*caches, wide[::3, :7], start, cu, cu, 200)
    want = four_bits(c.v[:100])[2] if bits == 4 else c.v[:100]
    assert torch.equal(v[:100].cpu(), want) and torch.equal(v[:100], v[100:]) and torch.equal(k[:100], k[100:])
