"""Shared-prefix attention against its definition in 64 bits: forward, backward, the
single-token form, refusals, streams and graphs."""

import ctypes
import math

import numpy as np
import pytest
import torch

import bwd_packed_varlen_gb300 as ta
import oracle
from prefix_common import prefix_check, prefix_plain, prefix_sums

gpu = pytest.mark.gpu
BR, TL, PAD = "padding_causal_bottom_right", "padding_causal", "padding"
FWD, ALL = ("out", "lse"), ("dq", "dk", "dv", "dkp", "dvp")


class Case:
    """Random inputs; every row that is no token holds +-1e3, and the rows behind the
    prefix's real length too."""

    def __init__(self, seed, lq, lk, prefix, hq, hkv, d, dtype, mask, prefix_rows=None, slot_q=3, slot_k=5, tail=2,
                 spread=0.0):
        gen = torch.Generator().manual_seed(seed)
        self.mask, self.dtype, self.scale, self.prefix = mask, dtype, 1.0 / math.sqrt(d), prefix
        rows = prefix if prefix_rows is None else prefix_rows
        sq, sk = ([(n + s - 1) // s * s for n in ls] for ls, s in ((lq, slot_q), (lk, slot_k)))
        oq, ok = np.cumsum([0] + sq), np.cumsum([0] + sk)
        self.spans_q, self.spans_k = list(zip(oq.tolist(), lq)), list(zip(ok.tolist(), lk))
        tq, tk = int(oq[-1]) + tail, int(ok[-1]) + tail
        wide = torch.exp(spread * torch.randn(d, generator=gen))

        def make(n, h, spans, w=1.0):
            x = torch.randn(n, h, d, generator=gen) * w
            real = torch.zeros(n, dtype=torch.bool)
            for o, m in spans:
                real[o:o + m] = True
            x[~real] = 1e3 * torch.sign(x[~real])
            return x.to(dtype)
        self.q, self.dout = make(tq, hq, self.spans_q, wide), make(tq, hq, self.spans_q)
        self.k, self.v = make(tk, hkv, self.spans_k), make(tk, hkv, self.spans_k)
        self.kp, self.vp = make(rows, hkv, [(0, prefix)]), make(rows, hkv, [(0, prefix)])
        self.cu = [prefix_sums(lq), prefix_sums(lk), torch.tensor(oq, dtype=torch.int32), torch.tensor(ok, dtype=torch.int32)]
        self.len = None if prefix_rows is None else torch.tensor([prefix], dtype=torch.int32)

    def dev(self):
        if not hasattr(self, "on"):
            self.on = [x.cuda() for x in (self.q, self.k, self.v, self.kp, self.vp)]
            self.cu_on = [c.cuda() for c in self.cu]
            self.len_on = None if self.len is None else self.len.cuda()
            self.dout_on = self.dout.cuda()
        return self

    def fwd(self, **kw):
        self.dev()
        return ta.prefix_fwd(*self.on, *self.cu_on, self.scale, self.mask, self.len_on, **kw)

    def bwd(self, out, lse, **kw):
        self.dev()
        return ta.prefix_bwd(*self.on, out, self.dout_on, lse, *self.cu_on, self.scale, self.mask, self.len_on, **kw)

    def plain(self, out_in=None):
        return prefix_plain(self.q, self.k, self.v, self.kp, self.vp, self.dout, self.spans_q, self.spans_k,
                            self.prefix, self.scale, self.mask, out_in)

    def check(self, backward=True):
        out, lse = self.fwd()
        ref = self.plain()
        prefix_check({"out": out, "lse": lse}, ref, FWD, self.dtype)
        if backward:
            grads = self.bwd(out, lse)
            prefix_check(dict(zip(ALL, grads)), ref, ALL, self.dtype)
        return out, lse


def _bits(ts):
    return [t.view(torch.int32 if t.dtype == torch.float32 else torch.int16).clone() for t in ts]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(_bits(a), _bits(b)))


# ------------------------------------------------------------------ on the CPU
def test_plain_form_against_the_packed_oracle():
    """With the padding mask the prefix is the first keys of every sequence, and with the
    lower-right triangle too (key j <= i + (P + Lk) - Lq): the packed oracle on joined keys
    gives the same, and its dk, dv split into the own and, summed, the prefix's."""
    for mask in (PAD, BR):
        c = Case(3, [4, 0, 7], [6, 2, 7], 5, 4, 2, 8, torch.float16, mask)
        ref = c.plain()
        K, V, spans, rows = [], [], [], 0
        for o, n in c.spans_k:
            K.append(torch.cat((c.kp, c.k[o:o + n])))
            V.append(torch.cat((c.vp, c.v[o:o + n])))
            spans.append((rows, 5 + n))
            rows += 5 + n
        f64 = [x.double().numpy() for x in (c.q, torch.cat(K), torch.cat(V), c.dout)]
        cuk = prefix_sums([n for _, n in spans]).numpy()
        got = oracle.attn_fwd_bwd_thd(*f64, c.cu[0].numpy(), cuk, c.cu[2].numpy(), cuk, c.scale, mask)
        got = got if not isinstance(got, dict) else [got[n] for n in ("out", "lse", "dq", "dk", "dv")]
        out, lse, dq, dk, dv = [torch.from_numpy(np.asarray(x)) for x in got[:5]]
        assert torch.allclose(ref["out"], out) and torch.allclose(ref["lse"], lse) and torch.allclose(ref["dq"], dq)
        for name, pre, x in (("dk", "dkp", dk), ("dv", "dvp", dv)):
            assert torch.allclose(ref[pre], sum(x[o:o + 5] for o, _ in spans))
            for (o, n), (oo, m) in zip(spans, c.spans_k):
                assert torch.allclose(ref[name][oo:oo + m], x[o + 5:o + n])


def test_plain_form_gradients_against_differences():
    """Central differences of sum(out * dout) in float64: error O(h^2)."""
    c = Case(4, [3, 2], [3, 2], 4, 2, 1, 8, torch.float16, TL, slot_q=1, slot_k=1, tail=0)
    t = {n: getattr(c, n).double() for n in ("q", "k", "v", "kp", "vp")}

    def loss(x):
        r = prefix_plain(x["q"], x["k"], x["v"], x["kp"], x["vp"], c.dout, c.spans_q, c.spans_k, 4, c.scale, TL)
        return (r["out"] * c.dout.double()).sum().item()
    ref = c.plain()
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("kp", "dkp"), ("vp", "dvp")):
        for i in (0, 11, t[name].numel() - 1):
            v = []
            for h in (1e-4, -1e-4):
                x = {**t, name: t[name].clone()}
                x[name].view(-1)[i] += h
                v.append(loss(x))
            assert abs((v[0] - v[1]) / 2e-4 - ref[grad].view(-1)[i].item()) < 1e-6


def test_refusals_launch_nothing():
    """Bad arguments return their code before any launch (placeholder pointers)."""
    lib = ta.library()
    P, odd, cu, big = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8), ctypes.c_void_p(1 << 21), ctypes.c_size_t(1 << 40)

    def fwd(t=(), plen=None, batch=2, tq=64, tk=64, rows=32, hq=4, hkv=2, d=64, scale=0.1, mask=1, dtype=1, ws=P,
            wsb=big, cus=(cu,) * 4):
        ptrs = [P] * 7
        for i, v in t:
            ptrs[i] = v
        return lib.te_attn_prefix_fwd_thd(*ptrs, *cus, plen, batch, tq, tk, rows, hq, hkv, d, scale, mask, dtype, ws, wsb, None)

    def bwd(t=(), plen=None, rows=32, wsb=big, hq=4):
        ptrs = [P] * 13
        for i, v in t:
            ptrs[i] = v
        return lib.te_attn_prefix_bwd_thd(*ptrs, cu, cu, cu, cu, plen, 2, 64, 64, rows, hq, 2, 64, 0.1, 1, 1, P, wsb, None)
    assert fwd(mask=4) == -2 and fwd(d=12) == -2 and fwd(d=264) == -2 and fwd(dtype=7) == -2
    assert fwd(hq=3) == -1 and fwd(batch=0) == -1 and fwd(rows=-1) == -1 and fwd(tq=-1) == -1
    assert fwd(scale=float("nan")) == -1 and fwd(ws=None) == -1 and fwd(cus=(cu, cu, None, cu)) == -1
    assert fwd(tq=1 << 30, hq=4) == -2                       # total_q * hq past 2^31
    assert fwd(wsb=ctypes.c_size_t(16)) == -3 and bwd(wsb=ctypes.c_size_t(16)) == -3
    assert fwd(plen=ctypes.c_void_p((1 << 20) + 2)) == -1    # prefix_len off its alignment
    for i in range(7):
        assert fwd(t=[(i, None)]) == -1, i
        if i != 6:                                           # lse needs no 16 bytes
            assert fwd(t=[(i, odd)]) == -1, i
    for i in range(13):
        assert bwd(t=[(i, None)]) == -1, i
        if i != 7:
            assert bwd(t=[(i, odd)]) == -1, i
    assert bwd(hq=5) == -1
    assert lib.te_attn_last_error()
    sizes = (2, 64, 64, 32, 4, 2, 64)
    assert ta.prefix_fwd_workspace_size(*sizes) > 0 and ta.prefix_bwd_workspace_size(*sizes) > 0
    assert ta.prefix_fwd_workspace_size(0, 64, 64, 32, 4, 2, 64) == 0
    assert ta.prefix_fwd_workspace_size(2, 64, 64, -1, 4, 2, 64) == 0
    assert ta.prefix_bwd_workspace_size(2, 64, 64, 32, 4, 3, 64) == 0
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c = prefix_sums([4])
    with pytest.raises(ValueError):
        ta.prefix_fwd(x, x, x, x, x, c, c, c, c, 0.1)
    with pytest.raises(ValueError):
        ta.shared_prefix_attention(x, x, x, x, x, c, c)


# ------------------------------------------------------------------ on the GPU
@gpu
@pytest.mark.parametrize("mask", [BR, TL, PAD])
@pytest.mark.parametrize("d,hq,hkv,dtype", [(128, 8, 2, torch.bfloat16), (64, 6, 1, torch.float16), (256, 4, 2, torch.bfloat16),
                                            (48, 3, 3, torch.bfloat16), (8, 2, 1, torch.float16), (200, 5, 1, torch.float16),
                                            (96, 12, 2, torch.bfloat16)])
def test_ragged(d, hq, hkv, dtype, mask):
    """Query lengths 0, 1 and past a tile, own keys absent, fewer than queries (rows before
    the triangle) and past a tile, a prefix that ends inside a tile, pad rows everywhere."""
    Case(d + len(mask), [1, 0, 37, 140, 5, 1], [9, 4, 37, 150, 0, 1], 133, hq, hkv, d, dtype, mask, spread=0.5).check()


@gpu
@pytest.mark.parametrize("prefix,rows", [(0, None), (0, 40), (1, None), (127, 300), (128, None), (129, 129), (700, None)])
def test_prefix_lengths(prefix, rows):
    """No prefix, one key, tile borders, and a real length on the device below the rows
    (whose gradients come out as zeros)."""
    Case(prefix + 1, [1, 3, 0, 70], [1, 20, 0, 70], prefix, 4, 2, 64, torch.bfloat16, BR, prefix_rows=rows).check()


@gpu
@pytest.mark.parametrize("d,hq,hkv,batch,prefix", [(128, 32, 8, 33, 1000), (64, 8, 8, 5, 4100), (256, 16, 2, 9, 513),
                                                   (128, 7, 1, 70, 257), (96, 40, 2, 3, 2049), (128, 136, 1, 2, 300)])
def test_single_tokens(d, hq, hkv, batch, prefix):
    """A decoding step: one query per sequence, caches of 0 to 900 keys in wider slots; a
    group of 136 heads fills more than a tile by itself."""
    lk = [(37 * i * i + 11 * i) % 900 for i in range(batch)]
    dtype = torch.float16 if batch % 2 else torch.bfloat16
    Case(batch, [1] * batch, lk, prefix, hq, hkv, d, dtype, BR, slot_q=1, slot_k=64, spread=0.4).check(backward=False)


@gpu
@pytest.mark.parametrize("d,hq,hkv,batch,longest", [(128, 8, 2, 84, 2600), (64, 4, 4, 150, 1500), (256, 16, 2, 40, 1900),
                                                    (80, 18, 2, 64, 1100)])
def test_many_long_caches(d, hq, hkv, batch, longest):
    """Decoding where every block goes through many items of many key tiles, on one stream and
    on both: groups of 1 to 8 heads and of 9; the same bits every time."""
    lk = [longest - (91 * i * i + 13 * i) % (longest // 2) for i in range(batch)]
    c = Case(batch, [1] * batch, lk, 700, hq, hkv, d, torch.bfloat16, BR, slot_q=1, slot_k=64, spread=0.4)
    out, lse = c.fwd()
    for _ in range(10):
        again = c.fwd()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    c.check(backward=False)


@gpu
def test_long_cache_of_one_sequence():
    """A single query over a long axis, which is split and joined; scores that grow along it
    move the running maximum in every part."""
    c = Case(12, [1], [9000], 5000, 4, 1, 64, torch.bfloat16, BR, slot_q=1)
    ramp = torch.linspace(0, 6, 5000)[:, None, None] * torch.sign(c.q[:1, :1].float())
    c.kp = (c.kp.float() + ramp / 2).to(c.dtype)
    c.check(backward=False)


@gpu
@pytest.mark.parametrize("d", [128, 256])
def test_scores_that_grow(d):
    """The running maximum moves in most key tiles, of the prefix and of the own keys, so that
    what is summed so far is scaled down again and again, while other rows' maxima stay."""
    c = Case(31, [1, 90], [700, 800], 1500, 4, 1, d, torch.float16, BR, slot_q=1)
    for x, n, b in ((c.kp, 1500, 0), (c.k[:700], 700, 0), (c.k[-802:-2], 800, 1)):
        o = c.spans_q[b][0]
        ramp = torch.linspace(0, 40.0 * n / 1500, n)[:, None, None]
        x += (ramp * torch.sign(c.q[o:o + 1, :1].float()) / math.sqrt(d)).to(c.dtype)
    c.check(backward=False)


@gpu
def test_large_scores_and_equal_scores():
    """Peaked softmaxes (scores of hundreds) and constant ones (every key alike)."""
    c = Case(13, [1, 40, 3], [30, 40, 300], 400, 4, 2, 128, torch.bfloat16, BR)
    c.scale = 4.0
    out, lse = c.fwd()
    # a score is a sum of 128 products rounded at 2^-24 of magnitudes up to 4 * 128 * 4, and lse follows it
    prefix_check({"out": out, "lse": lse}, c.plain(), FWD, c.dtype, lse_tol=2048 * 2.0 ** -24 * 16)
    c = Case(14, [1, 40, 3], [30, 40, 300], 400, 4, 2, 128, torch.bfloat16, BR)
    c.scale = 0.0
    c.check()


@gpu
def test_bad_lengths_are_reported():
    """A sequence whose real length exceeds its slot counts as empty and raises the status bit,
    as does a prefix length out of range; the other sequences keep their results."""
    c = Case(15, [2, 3, 4], [4, 5, 6], 50, 4, 2, 64, torch.bfloat16, BR, prefix_rows=64, slot_q=4, slot_k=8).dev()
    ws = torch.empty(ta.prefix_fwd_workspace_size(3, c.q.shape[0], c.k.shape[0], 64, 4, 2, 64), dtype=torch.uint8, device="cuda")
    good, _ = c.fwd(workspace=ws)
    assert ta.read_status(ws) == 0
    c.cu_on[0] = torch.tensor([0, 2, 11, 15], dtype=torch.int32).cuda()
    out, _ = c.fwd(workspace=ws)
    assert ta.read_status(ws) == 1
    assert torch.equal(out[:4], good[:4]) and torch.equal(out[8:], good[8:]) and torch.equal(out[4:8], torch.zeros_like(out[4:8]))
    c.cu_on[0], c.len_on = c.cu[0].cuda(), torch.tensor([65], dtype=torch.int32).cuda()
    out, lse = c.fwd(workspace=ws)
    assert ta.read_status(ws) == 1
    c.prefix = 0
    prefix_check({"out": out, "lse": lse}, c.plain(), FWD, c.dtype)
    wsb = torch.empty(ta.prefix_bwd_workspace_size(3, c.q.shape[0], c.k.shape[0], 64, 4, 2, 64), dtype=torch.uint8, device="cuda")
    c.bwd(out, lse, workspace=wsb)
    assert ta.read_status(wsb) == 1


@gpu
@pytest.mark.parametrize("d,hq,hkv,dtype", [(128, 8, 2, torch.bfloat16), (64, 3, 3, torch.float16), (256, 8, 1, torch.bfloat16)])
@pytest.mark.parametrize("mask", [BR, TL, PAD])
def test_forward_takes_any_bits_in_the_pads(d, hq, hkv, dtype, mask):
    """NaN and infinities in every row that holds no token, in a cache's free slots, behind the
    last sequence and behind the prefix's real length: the same bits as with zeros there."""
    c = Case(23, [1, 0, 37, 70, 1, 5], [9, 4, 37, 150, 0, 301], 133, hq, hkv, d, dtype, mask, prefix_rows=200, slot_k=64, tail=9).dev()
    spans = (c.spans_q, c.spans_k, c.spans_k, [(0, 133)], [(0, 133)])
    free = []
    for x, at in zip(c.on, spans):
        keep = torch.zeros(x.shape[0], dtype=torch.bool)
        for o, n in at:
            keep[o:o + n] = True
        free.append(~keep)
        x[free[-1].cuda()] = 0.0
    ref = c.fwd()
    for bad in (float("nan"), float("inf"), -float("inf")):
        for x, rows in zip(c.on, free):
            x[rows.cuda()] = bad
        assert _same(ref, c.fwd())


@gpu
def test_a_nan_is_not_hidden():
    """NaN in a key or value that a row sees comes out as NaN in that row, and only there."""
    c = Case(24, [1, 1, 40, 1], [30, 300, 40, 600], 200, 4, 2, 64, torch.bfloat16, BR).dev()
    (oq, _), (ok, _) = c.spans_q[1], c.spans_k[1]
    ref, _ = c.fwd()
    for x in (c.on[1], c.on[2]):
        x[ok + 270, 0, 5] = float("nan")
        out, lse = c.fwd()
        bad = torch.isnan(out).any(-1)
        assert bad[oq, :2].all() and not bad[oq, 2:].any() and int(bad.sum()) == 2
        assert torch.equal(out[oq + 1:].view(torch.int16), ref[oq + 1:].view(torch.int16))
    c.on[4][17, 1, 3] = float("nan")
    out, _ = c.fwd()
    rows = torch.zeros(out.shape[0], dtype=torch.bool)
    for o, n in c.spans_q:
        rows[o:o + n] = True
    assert torch.isnan(out[rows][:, 2:, 3]).all() and not torch.isnan(out[~rows]).any()


@gpu
@pytest.mark.parametrize("batch", [1100, 2100])
def test_many_sequences(batch):
    """More sequences than the scheduler has threads, and than offsets fit in shared memory."""
    lk = [(7 * i) % 40 for i in range(batch)]
    lq = [1 if i % 5 else i % 3 for i in range(batch)]
    Case(batch, lq, lk, 60, 2, 1, 64, torch.bfloat16, BR, slot_q=1, slot_k=4).check()


@gpu
def test_nothing_to_read_or_to_answer():
    """No own keys at all, no prefix either, no queries: zeros, -infinity, and gradients of zero."""
    for lq, lk, prefix, tail in (([1, 3], [0, 0], 50, 0), ([1, 3], [0, 0], 0, 0), ([0, 0], [4, 5], 30, 0), ([0, 0], [4, 5], 30, 3)):
        c = Case(25, lq, lk, prefix, 4, 2, 64, torch.float16, BR, slot_q=1, slot_k=1, tail=tail)
        if tail == 0 and sum(lk) == 0:
            assert c.k.shape[0] == 0
        out, lse = c.fwd()
        grads = c.bwd(out, lse)
        names = (FWD if c.q.shape[0] else ()) + ALL
        prefix_check({"out": out, "lse": lse, **dict(zip(ALL, grads))}, c.plain(), names, c.dtype)


@gpu
def test_overlapping_sequences_are_reported():
    """Offsets that fall back put two sequences on the same rows; with more tokens than rows
    nothing is computed, and the status says so."""
    c = Case(26, [40, 1, 40], [40, 8, 40], 50, 4, 2, 64, torch.bfloat16, BR, slot_q=1, slot_k=1, tail=0).dev()
    sizes = (3, c.q.shape[0], c.k.shape[0], 50, 4, 2, 64)
    ws = torch.empty(ta.prefix_fwd_workspace_size(*sizes), dtype=torch.uint8, device="cuda")
    c.cu_on[0] = prefix_sums([60, 0, 60]).cuda()
    c.cu_on[1] = prefix_sums([60, 0, 60]).cuda()
    c.cu_on[2] = torch.tensor([0, 81, 0, 81], dtype=torch.int32).cuda()
    c.cu_on[3] = torch.tensor([0, 88, 0, 88], dtype=torch.int32).cuda()
    out, lse = c.fwd(workspace=ws)
    assert ta.read_status(ws) == 1
    wsb = torch.empty(ta.prefix_bwd_workspace_size(*sizes), dtype=torch.uint8, device="cuda")
    out.zero_()
    lse.zero_()
    grads = c.bwd(out, lse, workspace=wsb)
    assert ta.read_status(wsb) == 1 and all(torch.equal(g, torch.zeros_like(g)) for g in grads)


@gpu
def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace, do not touch each other."""
    cs = [Case(s, [1] * 30, [(s + 41 * i) % 700 for i in range(30)], 900, 8, 2, 128, torch.bfloat16, BR).dev() for s in (27, 28)]
    refs = [[x.clone() for x in c.fwd()] for c in cs]
    grads = [[x.clone() for x in c.bwd(*r)] for c, r in zip(cs, refs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, (c, st) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(st):
                out, lse = c.fwd()
                got[i].append([out, lse, *c.bwd(out, lse)])
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert _same(refs[i] + grads[i], g)


@gpu
def test_given_outputs_and_streams():
    """Outputs that the caller gives come back as the same objects; a stream given by its handle
    is used for the launches and for what is allocated; keyword and positional forms agree."""
    c = Case(30, [1, 5, 1], [40, 5, 300], 200, 4, 2, 64, torch.bfloat16, BR).dev()
    out, lse = c.fwd()
    grads = c.bwd(out, lse)
    o, l = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
    got = ta.prefix_fwd(*c.on, *c.cu_on, c.scale, BR, None, o, l)
    assert got[0] is o and got[1] is l and _same((out, lse), got)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        a = c.fwd(stream=side.cuda_stream)
        b = c.bwd(*a, stream=side.cuda_stream)
        torch.empty(1 << 20, device="cuda").fill_(float("nan"))  # of the current stream's memory
        side.synchronize()
        assert _same((out, lse, *grads), (*a, *b))
    d = [torch.empty_like(x) for x in grads]
    got = ta.prefix_bwd(*c.on, out, c.dout_on, lse, *c.cu_on, c.scale, BR, None, *d)
    assert all(x is y for x, y in zip(got, d)) and _same(grads, got)
    assert not any(x.requires_grad for x in ta.prefix_fwd(c.on[0].clone().requires_grad_(), *c.on[1:], *c.cu_on, c.scale, BR))


@gpu
def test_arguments_that_do_not_fit_are_refused():
    """Shapes, types, strides and devices that do not go together, before any launch."""
    c = Case(29, [3, 1], [3, 9], 20, 4, 2, 64, torch.bfloat16, BR).dev()
    q, k, v, kp, vp = c.on
    cu = c.cu_on

    def call(tensors=c.on, lens=cu, **kw):
        with pytest.raises(ValueError):
            ta.prefix_fwd(*tensors, *lens, 0.1, **kw)
    call((q.float(), k, v, kp, vp))
    call((q, k.half(), v, kp, vp))
    call((q, k, v[:-1], kp, vp))
    call((q, k, v, kp[:, :1], vp[:, :1]))
    call((q, k, v, kp, vp[:-1]))
    call((q[..., :32], k, v, kp, vp))
    call((q.transpose(0, 1), k, v, kp, vp))
    call((q, k, v, kp.cpu(), vp))
    call(lens=(cu[0].long(), *cu[1:]))
    call(lens=(cu[0], cu[1][:-1], *cu[2:]))
    call(lens=(cu[0].cpu(), *cu[1:]))
    call(out=torch.empty_like(q)[:-1])
    call(lse=torch.empty(q.shape[:2], dtype=torch.float64, device="cuda"))
    call(prefix_len=torch.tensor([3, 4], dtype=torch.int32).cuda())
    call(mask_type="no_mask")
    with pytest.raises(RuntimeError):
        ta.prefix_fwd(*c.on, *cu, 0.1, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    out, lse = c.fwd()
    with pytest.raises(ValueError):
        ta.prefix_bwd(*c.on, out, c.dout_on.transpose(0, 1), lse, *cu, 0.1)
    with pytest.raises(ValueError):
        ta.prefix_bwd(*c.on, out, c.dout_on, lse.double(), *cu, 0.1)


@gpu
@pytest.mark.parametrize("shape", ["steps", "long"])
def test_bits_do_not_depend_on_what_was_there(shape):
    """Repeated calls, poisoned outputs and workspaces, other streams: the same bits."""
    c = (Case(16, [1] * 9, [5, 300, 0, 64, 700, 1, 128, 129, 33], 900, 8, 2, 128, torch.bfloat16, BR) if shape == "steps" else
         Case(17, [300, 1, 77, 513], [300, 9, 77, 600], 450, 8, 2, 128, torch.float16, BR)).dev()
    out, lse = c.fwd()
    first = [out, lse, *c.bwd(out, lse)]
    sizes = (len(c.spans_q), c.q.shape[0], c.k.shape[0], c.kp.shape[0], c.q.shape[1], c.k.shape[1], c.q.shape[2])
    for poison in (0xff, 0x7f):
        ws, wsb = (torch.full((n,), poison, dtype=torch.uint8, device="cuda") for n in
                   (ta.prefix_fwd_workspace_size(*sizes), ta.prefix_bwd_workspace_size(*sizes)))
        outs = [torch.full_like(x, float("nan")) for x in first]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.fwd(out=outs[0], lse=outs[1], workspace=ws)
            c.bwd(outs[0], outs[1], dq=outs[2], dk=outs[3], dv=outs[4], dk_prefix=outs[5], dv_prefix=outs[6], workspace=wsb)
        torch.cuda.synchronize()
        assert ta.read_status(ws) == 0 and ta.read_status(wsb) == 0
        assert _same(first, outs)


@gpu
def test_captured_steps_follow_their_buffers():
    """A captured forward and backward, replayed after the caches grew and the inputs changed."""
    c = Case(18, [1, 2, 1, 40], [10, 64, 3, 40], 200, 8, 2, 64, torch.bfloat16, BR, slot_k=128).dev()
    sizes = (4, c.q.shape[0], c.k.shape[0], 200, 8, 2, 64)
    ws, wsb = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in
               (ta.prefix_fwd_workspace_size(*sizes), ta.prefix_bwd_workspace_size(*sizes)))
    out, lse = c.fwd(workspace=ws)
    grads = c.bwd(out, lse, workspace=wsb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.fwd(out=out, lse=lse, workspace=ws)
        c.bwd(out, lse, workspace=wsb, **dict(zip(("dq", "dk", "dv", "dk_prefix", "dv_prefix"), grads)))
    c.cu_on[1].copy_(prefix_sums([11, 120, 90, 100]))
    gen = torch.Generator().manual_seed(1)
    for x in c.on[:3]:
        x.copy_(torch.randn(x.shape, generator=gen))
    for x in (out, lse, *grads):
        x.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    got = _bits([out, lse, *grads])
    out2, lse2 = c.fwd()
    assert all(torch.equal(a, b) for a, b in zip(got, _bits([out2, lse2, *c.bwd(out2, lse2)])))


@gpu
def test_debug_build_is_clean():
    """The bounds-checking build reports no offset outside a buffer, and the same bits."""
    for c in (Case(19, [1] * 5, [5, 300, 0, 64, 70], 400, 8, 2, 128, torch.bfloat16, BR),
              Case(20, [100, 0, 77, 1], [300, 9, 77, 1], 150, 4, 2, 256, torch.float16, TL)):
        out, lse = c.fwd()
        ref = [out, lse, *c.bwd(out, lse)]
        with ta.debug_build():
            sizes = (len(c.spans_q), c.q.shape[0], c.k.shape[0], c.kp.shape[0], c.q.shape[1], c.k.shape[1], c.q.shape[2])
            ws, wsb = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in
                       (ta.prefix_fwd_workspace_size(*sizes), ta.prefix_bwd_workspace_size(*sizes)))
            o, l = c.fwd(workspace=ws)
            got = [o, l, *c.bwd(o, l, workspace=wsb)]
            assert ta.read_status(ws) == 0 and ta.read_status(wsb) == 0
        assert _same(ref, got)


@gpu
def test_autograd_with_rotation():
    """The operators as they are used together: rotate q and k behind the prefix, attend,
    and go back to the unrotated leaves; compared with float64 through torch."""
    lq, P, hq, hkv, d = [9, 1, 30], 40, 4, 2, 64
    c = Case(21, lq, lq, P, hq, hkv, d, torch.bfloat16, TL)
    w, m = ta.rope_frequencies(32, scaling="yarn", factor=8.0, original_length=64)
    c.dev()
    leaves = [x.clone().requires_grad_() for x in c.on]
    q, k, v, kp, vp = leaves
    cu_q, cu_k, pad_q, pad_k = c.cu_on
    start = torch.full((3,), P, dtype=torch.int32, device="cuda")
    qr, _ = ta.rotary_positions(q, None, w, cu_q, pad_q, start, mscale=m)
    kr, _ = ta.rotary_positions(k, None, w, cu_k, pad_k, start, mscale=m)
    kpr, _ = ta.rotary_positions(kp, None, w, prefix_sums([P]).cuda(), mscale=m)
    out, lse = ta.shared_prefix_attention(qr, kr, v, kpr, vp, cu_q, cu_k, pad_q, pad_k, return_lse=True)
    assert out.shape == (c.q.shape[0], hq * d) and not lse.requires_grad
    out.backward(c.dout_on.view(out.shape))

    ref = [x.double().requires_grad_() for x in (c.q, c.k, c.v, c.kp, c.vp)]
    wc = w.cpu()

    def turn(x, pos):
        cos, sin = ((pos[:, None] * wc).cos() * m)[:, None], ((pos[:, None] * wc).sin() * m)[:, None]
        a, b, rest = x[..., :16], x[..., 16:32], x[..., 32:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)
    total = torch.zeros(())
    outs = torch.zeros(c.q.shape, dtype=torch.float64)
    kpt = turn(ref[3], torch.arange(P).double())
    for (oq, n), (ok, _) in zip(c.spans_q, c.spans_k):
        pos = P + torch.arange(n).double()
        Q, K = turn(ref[0][oq:oq + n], pos), torch.cat((kpt, turn(ref[1][ok:ok + n], pos)))
        V = torch.cat((ref[4], ref[2][ok:ok + n]))
        K, V = (x.repeat_interleave(hq // hkv, dim=1) for x in (K, V))
        S = torch.einsum("ihd,jhd->hij", Q, K) * c.scale
        S[:, torch.cat((torch.zeros(n, P, dtype=torch.bool), torch.ones(n, n, dtype=torch.bool).triu(1)), 1)] = -math.inf
        o = torch.einsum("hij,jhd->ihd", torch.softmax(S, -1), V)
        outs[oq:oq + n] = o.detach()
        total = total + (o * c.dout.double()[oq:oq + n]).sum()
    total.backward()
    # q and k are rounded once more (u of each, so of every score's terms): norms within 4 u
    u = 2.0 ** -8
    assert (out.detach().cpu().double().view(outs.shape) - outs).norm() <= 4 * u * outs.norm()
    for a, b in zip(leaves, ref):
        assert (a.grad.cpu().double() - b.grad).norm() <= 4 * u * b.grad.norm()
