"""Sweeps over sinks that are cut into parts (sequences of more than 16 query tiles), in the forms that
a caller may give them: sequence-major, over used workspaces, in the debug build, captured, by autograd."""

import math

import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from prefix_common import prefix_check, prefix_sums
from test_window import ALL, BR, TL, Case, _same
from window_common import window_plain

pytestmark = pytest.mark.gpu
WINDOWS = [(100, 4), (150, 140), (60, 300)]  # sinks in the first key tile, the first two, past those


def _workspace(c, fill):
    B, (tq, hq, d), (tk, hkv, _) = len(c.cu[0]) - 1, c.q.shape, c.k.shape
    n = ta.window_bwd_workspace_size(B, tq, tk, hq, hkv, d, c.window, c.sinks)
    assert n > ta.window_bwd_workspace_size(B, tq, tk, hq, hkv, d, c.window, 0)  # parts are kept
    return torch.full((n,), fill, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_sequence_major(d, window, sinks):
    """The packed layout's results, bit for bit, on the same tokens; they are the definition's."""
    S, B, hq, hkv = 2500, 3, 2, 1
    gen = torch.Generator().manual_seed(81)
    q, k, v, g = (torch.randn(S, B, h, d, generator=gen).to(torch.bfloat16).cuda() for h in (hq, hkv, hkv, hq))
    lens = [2500, 41, 2310]
    cu, full = prefix_sums(lens).cuda(), prefix_sums([S] * B).cuda()
    out, lse = ta.window_fwd_sbhd(q, k, v, cu, cu, 0.1, window, sinks)
    grads = ta.window_bwd_sbhd(q, k, v, out, g, lse, cu, cu, 0.1, window, sinks)
    flat = [x.transpose(0, 1).flatten(0, 1).contiguous() for x in (q, k, v, g)]
    o2, l2 = ta.window_fwd(*flat[:3], cu, cu, full, full, 0.1, window, sinks)
    g2 = ta.window_bwd(*flat[:3], o2, flat[3], l2, cu, cu, full, full, 0.1, window, sinks)
    for x, y in zip((out, lse, *grads), (o2, l2, *g2)):
        assert torch.equal(x.transpose(0, 1).flatten(0, 1), y)
    if d == 64:
        spans = [(S * i, n) for i, n in enumerate(lens)]
        prefix_check(dict(zip(ALL, (o2, l2, *g2))), window_plain(*flat, spans, spans, 0.1, TL, window, sinks), ALL, torch.bfloat16)


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("mask", [TL, BR])
def test_repeats_and_what_buffers_held(mask, window, sinks):
    c = Case(82, [2600, 70, 4300], [2600, 90, 4400], window, sinks, 4, 2, 64, torch.float16, mask).dev()
    out, lse = c.fwd()
    grads = c.bwd(out, lse)
    poison = lambda t: torch.full_like(t.view(torch.uint8), 255).view(t.dtype)  # noqa: E731
    for fill in (255, 0, 0x7F):
        ws = _workspace(c, fill)
        for _ in range(2):  # the second time over what the first one left
            again = c.bwd(out, lse, dq=poison(grads[0]), dk=poison(grads[1]), dv=poison(grads[2]), workspace=ws)
            assert _same(grads, again) and ta.read_status(ws) == 0
    # a workspace that another problem's parts lie in
    other = Case(83, [4300, 2600], [4300, 2700], window, sinks, 4, 2, 64, torch.float16, mask).dev()
    big = torch.empty(max(_workspace(c, 0).numel(), _workspace(other, 0).numel()), dtype=torch.uint8, device="cuda")
    other.bwd(*other.fwd(), workspace=big)
    assert _same(grads, c.bwd(out, lse, workspace=big)) and ta.read_status(big) == 0


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_debug_build_finds_nothing(d, window, sinks):
    c = Case(84, [2300, 1, 2500], [2400, 60, 90], window, sinks, 2, 1, d, torch.float16, TL).dev()
    out, lse = c.fwd()
    grads = c.bwd(out, lse)
    with ta.debug_build():
        ws = _workspace(c, 255)
        assert _same(grads, c.bwd(out, lse, workspace=ws)) and ta.read_status(ws) == 0


@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_graph_replays_follow_their_buffers(window, sinks):
    """Inputs, and lengths with another number of parts."""
    a, b = (Case(s, n, n, window, sinks, 2, 1, 128, torch.bfloat16, TL, slot_q=1, slot_k=1, tail=0).dev()
            for s, n in ((85, [2600, 4300]), (86, [4500, 2400])))
    a.bwd(*a.fwd())
    want = [(*x, *b.bwd(*x)) for x in (b.fwd(),)][0]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = a.fwd()
        grads = a.bwd(out, lse)
    for x, y in zip(a.on + [a.dout_on] + a.cu_on, b.on + [b.dout_on] + b.cu_on):
        x.copy_(y)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert _same((out, lse, *grads), want)


@pytest.mark.parametrize("fmt", ["thd", "bshd", "sbhd"])
def test_autograd(fmt):
    B, S, hq, hkv, d = 2, 2300, 2, 1, 64
    gen = torch.Generator().manual_seed(87)
    q, k, v, g = (torch.randn(B, S, h, d, generator=gen).to(torch.float16) for h in (hq, hkv, hkv, hq))
    spans = [(0, 2300), (2300, 2200)]
    ref = window_plain(*(x.flatten(0, 1) for x in (q, k, v, g)), spans, spans, 1 / math.sqrt(d), TL, 90, 140)
    lay = {"thd": lambda x: x.flatten(0, 1), "bshd": lambda x: x, "sbhd": lambda x: x.transpose(0, 1)}[fmt]
    leaves = [lay(x).contiguous().cuda().requires_grad_() for x in (q, k, v)]
    cu, full = prefix_sums([2300, 2200]).cuda(), prefix_sums([S, S]).cuda()
    kw = {"cu_seqlens_q_padded": full, "cu_seqlens_kv_padded": full} if fmt == "thd" else {}
    out = ta.DotProductAttention(hq, d, hkv, qkv_format=fmt, window=90, sinks=140)(*leaves, cu, cu, **kw)
    grads = torch.autograd.grad(out, leaves, lay(g).reshape(out.shape).cuda())
    back = {"thd": lambda x: x, "bshd": lambda x: x.flatten(0, 1), "sbhd": lambda x: x.transpose(0, 1).flatten(0, 1)}[fmt]
    got = {n: back(x.detach().view(lay(y).shape)) for n, x, y in zip(("out", "dq", "dk", "dv"), (out, *grads), (q, q, k, v))}
    prefix_check(got, ref, ("out", "dq", "dk", "dv"), torch.float16)
