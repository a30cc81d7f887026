"""Sliding-window attention with sinks against its definition in 64 bits: forward, backward, both
layouts, the autograd path, refusals, graphs."""

import ctypes
import math

import numpy as np
import pytest
import torch

import bwd_packed_varlen_gb300 as ta
import oracle
from prefix_common import prefix_check, prefix_sums
from window_common import visible, window_plain

gpu = pytest.mark.gpu
BR, TL, PAD = "padding_causal_bottom_right", "padding_causal", "padding"
ALL = ("out", "lse", "dq", "dk", "dv")
FAR = 2 ** 31 - 1


class Case:
    """Random inputs; every row that is no token holds +-1e3."""

    def __init__(self, seed, lq, lk, window, sinks, hq, hkv, d, dtype, mask, slot_q=3, slot_k=5, tail=2):
        gen = torch.Generator().manual_seed(seed)
        self.mask, self.dtype, self.scale, self.window, self.sinks = mask, dtype, 1.0 / math.sqrt(d), window, sinks
        sq, sk = ([(n + s - 1) // s * s for n in ls] for ls, s in ((lq, slot_q), (lk, slot_k)))
        oq, ok = np.cumsum([0] + sq), np.cumsum([0] + sk)
        self.spans_q, self.spans_k = list(zip(oq.tolist(), lq)), list(zip(ok.tolist(), lk))
        tq, tk = int(oq[-1]) + tail, int(ok[-1]) + tail

        def make(n, h, spans):
            x = torch.randn(n, h, d, generator=gen)
            real = torch.zeros(n, dtype=torch.bool)
            for o, m in spans:
                real[o:o + m] = True
            x[~real] = 1e3 * torch.sign(x[~real])
            return x.to(dtype)
        self.q, self.dout = make(tq, hq, self.spans_q), make(tq, hq, self.spans_q)
        self.k, self.v = make(tk, hkv, self.spans_k), make(tk, hkv, self.spans_k)
        self.cu = [prefix_sums(lq), prefix_sums(lk), torch.tensor(oq, dtype=torch.int32), torch.tensor(ok, dtype=torch.int32)]

    def dev(self):
        if not hasattr(self, "on"):
            self.on = [x.cuda() for x in (self.q, self.k, self.v)]
            self.cu_on = [c.cuda() for c in self.cu]
            self.dout_on = self.dout.cuda()
        return self

    def fwd(self, **kw):
        self.dev()
        return ta.window_fwd(*self.on, *self.cu_on, self.scale, self.window, self.sinks, self.mask, **kw)

    def bwd(self, out, lse, **kw):
        self.dev()
        return ta.window_bwd(*self.on, out, self.dout_on, lse, *self.cu_on, self.scale, self.window, self.sinks, self.mask, **kw)

    def plain(self, out_in=None):
        return window_plain(self.q, self.k, self.v, self.dout, self.spans_q, self.spans_k, self.scale, self.mask, self.window,
                            self.sinks, out_in)

    def check(self):
        out, lse = self.fwd()
        got = dict(zip(ALL, (out, lse, *self.bwd(out, lse))))
        prefix_check(got, self.plain(), ALL, self.dtype)
        return got


def _bits(ts):
    return [t.view(torch.int32 if t.dtype == torch.float32 else torch.int16).clone() for t in ts]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(_bits(a), _bits(b)))


# ------------------------------------------------------------------ on the CPU
def test_plain_form_against_the_packed_oracle():
    """A window as long as the sequences leaves what the causal masks leave."""
    for mask in (TL, BR):
        c = Case(3, [4, 0, 7], [6, 2, 7], 100, 0, 4, 2, 8, torch.float16, mask)
        ref = c.plain()
        f64 = [x.double().numpy() for x in (c.q, c.k, c.v, c.dout)]
        got = oracle.attn_fwd_bwd_thd(*f64, *[x.numpy() for x in c.cu], c.scale, mask)
        got = got if not isinstance(got, dict) else [got[n] for n in ALL]
        for name, x in zip(ALL, got):
            assert torch.allclose(ref[name], torch.from_numpy(np.asarray(x))), name


def test_visible_keys_by_hand():
    assert visible(4, 4, TL, 2, 0).int().tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [0, 1, 1, 0], [0, 0, 1, 1]]
    assert visible(4, 4, TL, 1, 1).int().tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 0, 1]]
    assert visible(2, 4, BR, 2, 0).int().tolist() == [[0, 1, 1, 0], [0, 0, 1, 1]]
    assert visible(4, 2, TL, 2, 0).int().tolist() == [[1, 0], [1, 1], [0, 1], [0, 0]]
    assert visible(3, 1, BR, 5, 2).int().tolist() == [[0], [0], [1]]


def test_plain_form_gradients_against_differences():
    """Central differences of sum(out * dout) in float64: error O(h^2)."""
    c = Case(4, [5, 2], [5, 4], 2, 1, 2, 1, 8, torch.float16, TL, slot_q=1, slot_k=1, tail=0)
    ref, h = c.plain(), 1e-5
    t = {n: getattr(c, n).double() for n in ("q", "k", "v")}

    def loss(x):
        r = window_plain(x["q"], x["k"], x["v"], c.dout, c.spans_q, c.spans_k, c.scale, TL, 2, 1)
        return (r["out"] * c.dout.double()).sum().item()
    gen = torch.Generator().manual_seed(0)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        step = torch.randn(t[name].shape, generator=gen, dtype=torch.float64)
        up, down = ({**t, name: t[name] + s * h * step} for s in (1, -1))
        assert abs((loss(up) - loss(down)) / (2 * h) - (ref[grad] * step).sum().item()) < 1e-6


def _call(name, window, sinks, mask=2, rows=64, batch=1):
    """The entry point with addresses that are never looked at: its checks come first."""
    L, one = ta.library(), ctypes.c_void_p(4096)
    f32, null = ctypes.c_float(0.1), None
    cus = 4 if name.endswith("thd") else 2
    tensors = 5 if "fwd" in name else 9
    fn = getattr(L, "te_attn_" + name)
    return fn(*([one] * (tensors + cus)), batch, rows, rows, 2, 2, 64, f32, mask, window, sinks, 1, null, 0, null)


@pytest.mark.parametrize("name", ["window_fwd_thd", "window_bwd_thd", "window_fwd_sbhd", "window_bwd_sbhd"])
def test_refusals(name):
    last = lambda: ta.library().te_attn_last_error().decode()  # noqa: E731
    for window, sinks, mask, rows, code, word in ((0, 0, 2, 64, -1, "window"), (-5, 0, 3, 64, -1, "window"), (4, -1, 2, 64, -1, "sinks"),
                                                  (4, 0, 1, 64, -2, "causal"), (4, 0, 2, 2 ** 30, -2, "2^30"), (4, 0, 7, 64, -2, "mask_type"),
                                                  (4, 0, 2, 64, -1, "workspace")):
        assert _call(name, window, sinks, mask, rows) == code and word in last(), (window, sinks, mask, rows, last())


def test_refusals_in_python():
    q, cu = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ta.window_fwd(q, q, q, cu, cu, cu, cu, 0.1, 4)
    with pytest.raises(ValueError, match="tensor"):
        ta.window_fwd(q, None, q, cu, cu, cu, cu, 0.1, 4)
    with pytest.raises(ValueError, match="padded"):
        ta.window_fwd(q, q, q, cu, cu, None, cu, 0.1, 4)
    with pytest.raises(ValueError, match="window"):
        ta.dot_product_attention(q, q, q, cu, cu, sinks=3)
    with pytest.raises(ValueError, match="window"):
        ta.DotProductAttention(2, 64, sinks=3)


# ------------------------------------------------------------------ on the GPU
CASES = [
    # lq, lk, window, sinks, hq, hkv, d, dtype, mask
    ([40, 0, 1, 33], None, 7, 2, 4, 2, 64, torch.bfloat16, TL),
    ([300, 129], None, 64, 4, 2, 1, 64, torch.float16, TL),
    ([700, 5, 257], None, 128, 0, 2, 2, 128, torch.bfloat16, TL),
    ([700, 128], None, 129, 130, 4, 1, 128, torch.float16, TL),
    ([513, 640], None, 1, 0, 2, 2, 64, torch.bfloat16, TL),
    ([513, 127], None, 1, 1, 2, 1, 128, torch.bfloat16, BR),
    ([900], None, 200, 300, 2, 1, 80, torch.bfloat16, TL),
    ([130, 257, 1], [700, 300, 1000], 100, 4, 4, 2, 128, torch.bfloat16, BR),
    ([130, 257, 1], [700, 300, 1000], 100, 0, 2, 2, 64, torch.float16, BR),
    ([1, 2, 3], [900, 513, 129], 256, 5, 3, 1, 96, torch.float16, BR),
    ([600, 300], [10, 200], 50, 0, 2, 1, 64, torch.bfloat16, TL),   # rows behind the keys see none
    ([600, 300], [10, 0], 50, 3, 2, 1, 128, torch.bfloat16, TL),    # or the sinks alone
    ([600, 300], [10, 150], 50, 0, 2, 1, 128, torch.float16, BR),   # rows before the triangle
    ([260, 400], None, 90, 2, 2, 1, 256, torch.bfloat16, TL),
    ([70, 400], [500, 410], 131, 0, 2, 2, 256, torch.float16, BR),
    ([500, 20], [30, 20], 17, 0, 1, 1, 192, torch.bfloat16, TL),
    ([500], None, 3, 0, 1, 1, 8, torch.float16, TL),
    ([1200], None, 385, 1, 2, 1, 128, torch.bfloat16, TL),
    # sweeps over sinks that are cut into parts: more than 16 query tiles
    ([5000, 300, 2500], None, 100, 4, 2, 1, 64, torch.bfloat16, TL),
    ([2700], None, 300, 200, 2, 2, 128, torch.float16, TL),
    ([2600], None, 64, 140, 1, 1, 256, torch.bfloat16, TL),
    ([2500, 4300], [6000, 4400], 90, 3, 2, 1, 64, torch.float16, BR),   # the sinks lie before every window
    ([4500], [60], 40, 20, 1, 1, 64, torch.bfloat16, TL),              # a single, short key tile
    ([4500], [900], 2300, 300, 1, 1, 64, torch.float16, BR),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_against_the_definition(case):
    lq, lk, *rest = case
    Case(11, lq, lq if lk is None else lk, *rest).check()


@gpu
@pytest.mark.parametrize("seed", range(12))
def test_random(seed):
    r = np.random.default_rng(1000 + seed)
    n = int(r.integers(1, 6))
    lq = [int(x) for x in r.integers(0, 420, n)]
    lk = [max(0, a + int(b)) for a, b in zip(lq, r.integers(-100, 400, n))]
    hkv = int(r.integers(1, 3))
    Case(seed, lq, lk, int(2 ** r.uniform(0, 9)), int(r.choice([0, 0, 1, 4, 60, 200])), hkv * int(r.integers(1, 5)), hkv,
         8 * int(r.integers(1, 33)), [torch.bfloat16, torch.float16][seed % 2], [TL, BR][int(r.integers(2))]).check()


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [-0.9, 0.0])
def test_other_scales(d, scale):
    """Negative ones, with scores far apart, and none at all. (Scores of a few tens: fp32's 2^-24 of
    them, and of the products in them, stays below the lse's 1e-4.)"""
    c = Case(12, [300, 40], [300, 60], 90, 3, 2, 1, d, torch.bfloat16, BR)
    c.scale = scale
    c.check()


@gpu
@pytest.mark.parametrize("mask", [TL, BR])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_windows_are_the_causal_masks(mask, d):
    """Window and sinks that leave everything: the entry points without them, bit for bit."""
    for window, sinks in ((FAR, 0), (1500, 3), (1, FAR), (1, 1000)):
        c = Case(5, [700, 1, 300], [900, 40, 300], window, sinks, 4, 2, d, torch.bfloat16, mask).dev()
        out, lse = c.fwd()
        same = ta.fwd(*c.on, *c.cu_on, c.scale, mask)
        assert _same((out, lse), same)
        assert _same(c.bwd(out, lse), ta.bwd(*c.on, out, c.dout_on, lse, *c.cu_on, c.scale, mask))


@gpu
def test_repeats_and_what_buffers_held():
    c = Case(6, [500, 77, 0, 300], [500, 200, 3, 40], 60, 3, 4, 2, 128, torch.bfloat16, TL).dev()
    first = c.fwd()
    grads = c.bwd(*first)
    poison = lambda t: torch.full_like(t.view(torch.uint8), 255).view(t.dtype)  # noqa: E731
    B, tq, hq, d = len(c.cu[0]) - 1, c.q.shape[0], 4, 128
    ws = torch.full((ta.window_bwd_workspace_size(B, tq, c.k.shape[0], hq, 2, d, 60, 3),), 255, dtype=torch.uint8, device="cuda")
    again = c.fwd(out=poison(first[0]), lse=poison(first[1]), workspace=ws)
    assert _same(first, again) and ta.read_status(ws) == 0
    ws.fill_(255)
    more = c.bwd(*first, dq=poison(grads[0]), dk=poison(grads[1]), dv=poison(grads[2]), workspace=ws)
    assert _same(grads, more) and ta.read_status(ws) == 0


@gpu
def test_debug_build_finds_nothing():
    for d in (128, 256):
        c = Case(7, [300, 1, 129], [400, 60, 5], 77, 2, 2, 1, d, torch.float16, TL).dev()
        out, lse = c.fwd()
        grads = c.bwd(out, lse)
        with ta.debug_build():
            ws = torch.empty(ta.window_bwd_workspace_size(3, c.q.shape[0], c.k.shape[0], 2, 1, d, 77, 2), dtype=torch.uint8, device="cuda")
            assert _same((out, lse), c.fwd(workspace=ws)) and ta.read_status(ws) == 0
            assert _same(grads, c.bwd(out, lse, workspace=ws)) and ta.read_status(ws) == 0


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_sequence_major(d):
    """The packed layout's results, bit for bit, on the same tokens."""
    S, B, hq, hkv = 300, 3, 4, 2
    gen = torch.Generator().manual_seed(8)
    q, k, v, g = (torch.randn(S, B, h, d, generator=gen).to(torch.bfloat16).cuda() for h in (hq, hkv, hkv, hq))
    cu, full = prefix_sums([300, 41, 130]).cuda(), prefix_sums([S] * B).cuda()
    out, lse = ta.window_fwd_sbhd(q, k, v, cu, cu, 0.1, 70, 3)
    grads = ta.window_bwd_sbhd(q, k, v, out, g, lse, cu, cu, 0.1, 70, 3)
    flat = [x.transpose(0, 1).flatten(0, 1).contiguous() for x in (q, k, v, g)]
    o2, l2 = ta.window_fwd(*flat[:3], cu, cu, full, full, 0.1, 70, 3)
    g2 = ta.window_bwd(*flat[:3], o2, flat[3], l2, cu, cu, full, full, 0.1, 70, 3)
    for x, y in zip((out, lse, *grads), (o2, l2, *g2)):
        assert torch.equal(x.transpose(0, 1).flatten(0, 1), y)


@gpu
@pytest.mark.parametrize("fmt", ["thd", "bshd", "sbhd"])
def test_autograd(fmt):
    B, S, hq, hkv, d = 2, 200, 4, 2, 64
    gen = torch.Generator().manual_seed(9)
    q, k, v, g = (torch.randn(B, S, h, d, generator=gen).to(torch.float16) for h in (hq, hkv, hkv, hq))
    spans = [(0, 200), (200, 150)]
    ref = window_plain(*(x.flatten(0, 1) for x in (q, k, v, g)), spans, spans, 1 / math.sqrt(d), TL, 50, 2)
    lay = {"thd": lambda x: x.flatten(0, 1), "bshd": lambda x: x, "sbhd": lambda x: x.transpose(0, 1)}[fmt]
    leaves = [lay(x).contiguous().cuda().requires_grad_() for x in (q, k, v)]
    cu = prefix_sums([200, 150]).cuda()
    kw = {"cu_seqlens_q_padded": prefix_sums([S, S]).cuda(), "cu_seqlens_kv_padded": prefix_sums([S, S]).cuda()} if fmt == "thd" else {}
    m = ta.DotProductAttention(hq, d, hkv, qkv_format=fmt, window=50, sinks=2)
    out = m(*leaves, cu, cu, **kw)
    # a gradient that starts off a 16-byte boundary
    dout = torch.empty(out.numel() + 1, dtype=torch.float16, device="cuda")[1:].view(out.shape)
    dout.copy_(lay(g).reshape(out.shape))
    grads = torch.autograd.grad(out, leaves, dout, retain_graph=True)
    back = {"thd": lambda x: x, "bshd": lambda x: x.flatten(0, 1), "sbhd": lambda x: x.transpose(0, 1).flatten(0, 1)}[fmt]
    got = {n: back(x.detach().view(lay(y).shape)) for n, x, y in zip(("out", "dq", "dk", "dv"), (out, *grads), (q, q, k, v))}
    prefix_check(got, ref, ("out", "dq", "dk", "dv"), torch.float16)
    again = torch.autograd.grad(out, leaves, dout, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    with pytest.raises(RuntimeError, match="second derivatives"):
        again[0].float().sum().backward()


@gpu
def test_graph_replays_follow_their_buffers():
    a, b = (Case(s, [300, 40], [300, 40], 33, 2, 2, 1, 64, torch.bfloat16, TL).dev() for s in (21, 22))
    a.bwd(*a.fwd())
    want = [(*x, *b.bwd(*x)) for x in (b.fwd(),)][0]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = a.fwd()
        grads = a.bwd(out, lse)
    for x, y in zip(a.on + [a.dout_on], b.on + [b.dout_on]):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert _same((out, lse, *grads), want)


@gpu
def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace, do not touch each other."""
    cs = [Case(s, [2600, 90, 300], [2600, 400, 300], 100, 3, 4, 2, 64, torch.bfloat16, BR).dev() for s in (31, 32)]
    refs = [[x.clone() for x in c.fwd()] for c in cs]
    grads = [[x.clone() for x in c.bwd(*r)] for c, r in zip(cs, refs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, (c, st) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(st):
                out, lse = c.fwd()
                got[i].append([out, lse, *c.bwd(out, lse)])
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert _same(refs[i] + grads[i], g)


@gpu
def test_given_outputs_streams_and_workspaces():
    c = Case(33, [5, 300, 1], [40, 300, 90], 50, 2, 4, 2, 128, torch.float16, BR).dev()
    out, lse = c.fwd()
    grads = c.bwd(out, lse)
    o, l = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
    got = c.fwd(out=o, lse=l)
    assert got[0] is o and got[1] is l and _same((out, lse), got)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        a = c.fwd(stream=side.cuda_stream)
        b = c.bwd(*a, stream=side.cuda_stream)
        torch.empty(1 << 20, device="cuda").fill_(float("nan"))  # of the current stream's memory
        side.synchronize()
        assert _same((out, lse, *grads), (*a, *b))
    for call, bad in ((c.fwd, dict(out=o[:-1])), (c.fwd, dict(lse=l.half())), (lambda **kw: c.bwd(out, lse, **kw), dict(dq=o.float())),
                      (lambda **kw: c.bwd(out, lse, **kw), dict(dk=o))):
        with pytest.raises(ValueError):
            call(**bad)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(ta.TeAttnError, match="workspace"):
        c.fwd(workspace=small)
    with pytest.raises(ta.TeAttnError, match="workspace"):
        c.bwd(out, lse, workspace=small)
    with pytest.raises(ValueError):
        ta.window_fwd(c.on[0].transpose(0, 1), *c.on[1:], *c.cu_on, c.scale, 50, 2)


@gpu
def test_a_captured_backward_of_its_own_leaves():
    """Forward and backward through autograd, captured into a graph, follow their leaves."""
    gen = torch.Generator().manual_seed(34)
    x = [torch.randn(260, h, 64, generator=gen).to(torch.bfloat16).cuda() for h in (4, 2, 2, 4)]
    cu = prefix_sums([200, 60]).cuda()

    def run(leaves):
        out = ta.dot_product_attention(*leaves, cu, cu, cu, cu, window=40, sinks=1)
        return (out.detach(), *torch.autograd.grad(out, leaves, x[3].view(260, -1)))
    want = run([t.clone().requires_grad_() for t in x[:3]])
    leaves = [torch.zeros_like(t).requires_grad_() for t in x[:3]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(leaves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(leaves)
    with torch.no_grad():
        for a, b in zip(leaves, x):
            a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert _same(want, got)
