"""Paged calls whose padded offsets fall back: the sequences that are consistent by themselves keep
their tokens, the others count as empty, and the status says so."""

import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from paged_common import places
from prefix_common import prefix_check
from test_paged_attention import BF, BR, FP
from test_paged_attention import Case as Attention
from test_paged_cache import Case as Cache
from window_common import window_plain

gpu = pytest.mark.gpu
PADDED = [60, 100, 10, 20]  # of three sequences; the second one's rows end before they begin
OFF, TOTAL = [60, 100, 10], 110


def _moved(c, like):
    """The case's sequences at OFF in rows that hold 1e3 elsewhere, `like` at the old offsets."""
    y = torch.full((TOTAL, *like.shape[1:]), 1e3).to(like.dtype)
    for old, new, n in zip(c.off, OFF, c.lengths):
        y[new:new + n] = like[old:old + n]
    return y


@gpu
@pytest.mark.parametrize("hq", [4, 160])  # 160: many rows a kv head, joined a head of a sequence at a time
@pytest.mark.parametrize("bits", [16, 4])
def test_attention(bits, hq):
    c = Attention(61, [30, 0, 8], [300, 5, 40], 16, hq, 2, 64, BF, bits)
    c.q, c.off, c.total = _moved(c, c.q), OFF, TOTAL
    c.cu[1] = torch.tensor(PADDED, dtype=torch.int32)
    ws = c.workspace()
    out, lse = c.fwd(out=torch.full_like(c.q, float("nan")).cuda(), lse=torch.full((TOTAL, hq), float("nan"), device="cuda"), workspace=ws)
    assert ta.read_status(ws) == 1
    ref = window_plain(c.q, *c.kv, None, list(zip(OFF, c.lengths)), list(zip(c.offk, c.keys)), c.scale, BR, 0, 0)
    prefix_check({"out": out, "lse": lse}, ref, ("out", "lse"), BF)


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_append_and_gather(bits):
    c = Cache(62, [30, 0, 8], [20, 5, 40], 16, 3, 2, 64, FP, bits, 64, fused=False)
    sound = c.fresh()
    q = c.append(sound).cpu()
    kv = [x.cpu() for x in c.gather(sound)]
    d = Cache(62, [30, 0, 8], [20, 5, 40], 16, 3, 2, 64, FP, bits, 64, fused=False)
    d.q, d.k, d.v = (_moved(c, x) for x in (c.q, c.k, c.v))
    d.total, d.cu[1] = TOTAL, torch.tensor(PADDED, dtype=torch.int32)
    caches, status = d.fresh(), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = [d.append(caches, status=status).cpu()]
    flat = lambda cs: [t for x in cs for t in (x if bits == 4 else (x,))]  # noqa: E731
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(flat(sound), flat(caches)))
    got += [x.cpu() for x in d.gather(caches)]
    for x, y in zip(got, (q, *kv)):
        want = _moved(c, y)
        rows, _, _ = places(d.table, 16, d.past, d.lengths, OFF)
        want[[r for r in range(TOTAL) if r not in rows.tolist()]] = 0
        assert torch.equal(x, want)


@gpu
@pytest.mark.parametrize("hq", [4, 160])
@pytest.mark.parametrize("bits", [16, 4])
def test_an_offset_far_below_zero(bits, hq):
    """The span from 5 to -2^31 is long as a 32-bit difference, and holds nothing."""
    c = Attention(63, [20, 0, 30], [3, 0, 9], 16, hq, 2, 64, BF, bits, slot=1, tail=20).dev()
    ws = c.workspace()
    bad = torch.tensor([5, -2 ** 31, 20, 70], dtype=torch.int32, device="cuda")
    kw = dict(out=torch.full_like(c.on[0], float("nan")), lse=torch.full((70, hq), float("nan"), device="cuda"), workspace=ws)
    out, lse = ta.paged_fwd(*c.on[:6], bad, c.scale, **kw)
    assert ta.read_status(ws) == 1
    spans = [(0, 0), (0, 0), (20, 30)]
    ref = window_plain(c.q, *c.kv, None, spans, list(zip(c.offk, c.keys)), c.scale, BR, 0, 0)
    prefix_check({"out": out, "lse": lse}, ref, ("out", "lse"), BF)


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_sequences_without_rows_are_reported(bits):
    """Inconsistent lengths, or a past below zero, of a sequence that has no row to be found by."""
    c = Cache(64, [5, 0, 4], [20, 7, 40], 16, 3, 2, 64, FP, bits, 64, slot=1, tail=0).dev()
    sound, status = c.fresh(), torch.zeros(1, dtype=torch.int32, device="cuda")
    q = c.append(sound, status=status)
    kv = c.gather(sound, status=status)
    assert status.item() == 0
    flat = lambda cs: [t for x in cs for t in (x if bits == 4 else (x,))]  # noqa: E731
    cu, past = c.cu_on[0], c.past_on
    for bad in ((torch.tensor([0, 5, 8, 12], dtype=torch.int32).cuda(), past), (cu, torch.tensor([20, -1, 40], dtype=torch.int32).cuda())):
        c.cu_on[0], c.past_on = bad
        caches = c.fresh()
        assert torch.equal(q, c.append(caches, status=status)) and status.item() == 1
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(flat(sound), flat(caches)))
        assert all(torch.equal(a, b) for a, b in zip(kv, c.gather(caches, status=status))) and status.item() == 1
