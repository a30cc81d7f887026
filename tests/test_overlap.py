"""Padded offsets that fall back put sequences on the same rows. They can then have more tiles than
a workspace of the call's sizes has room for: such a call computes nothing, says so in its status
and leaves zeros, and no byte outside its workspace is touched."""

import numpy as np
import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from prefix_common import prefix_sums

gpu = pytest.mark.gpu
BEHIND = 4096  # bytes behind a workspace that a call may not touch


def room_for_tiles(batch, rows, kv_rows, hkv=1, d=64):
    """Query tiles that a backward's workspace holds: two fp32 rows of 128 for each, per head."""
    one, two = (ta.bwd_workspace_size(batch, rows, kv_rows, hq, hkv, d) for hq in (1, 2))
    return (two - one) // (2 * 128 * 4)


def falling(batch, rows, times=1 << 30):
    """Offsets 0, rows, 0, rows, ...: every other sequence has all rows, those between have none left, up
    to the last of `times` sequences; those behind it are empty."""
    return torch.tensor([rows * (i % 2 if i < 2 * times else 1) for i in range(batch + 1)], dtype=torch.int32)


SWEEP = 16  # query tiles of a part of a cut sweep, for windows below 15 tiles


def parts_of(n, m, window, sinks, low):
    """Partial sums that a windowed backward keeps of a sequence of n queries and m keys: for each of the
    first two key tiles with a sink whose sweep ends more than a part behind its beginning, that beginning
    and the parts behind it (low: the lower-right mask)."""
    diag, total = m - n if low else 0, 0
    seen = min(m, max(0, n + diag)) if n else 0
    for kt in range(min(2, (min(sinks, seen) + 127) // 128)):
        first = max(0, kt * 128 - diag) // 128
        last = min(n, min(kt * 128 + 128, m) - 1 - diag + window)
        end = max((max(last, 0) + 127) // 128, first + SWEEP)
        left = (n + 127) // 128 - end
        total += (left + SWEEP - 1) // SWEEP + 1 if left > 0 else 0
    return total


def room_for_parts(batch, rows, kv_rows, window, sinks):
    """Partial sums that the workspace holds: at one head of 8 columns, 8 KB each and their entry."""
    sizes = (batch, rows, kv_rows, 1, 1, 8, window)
    extra = ta.window_bwd_workspace_size(*sizes, sinks) - ta.window_bwd_workspace_size(*sizes, 0)
    return max(0, extra - 4 * (batch + 1) - 3 * 256) // (8192 + 16)


class Overlap:
    def __init__(self, batch=19, rows=1300, kv_rows=260, hq=4, hkv=2, d=64, dtype=torch.bfloat16, times=None):
        gen = torch.Generator().manual_seed(51)
        self.sizes = (batch, rows, kv_rows, hq, hkv, d)
        times = (batch + 1) // 2 if times is None else times
        self.q, self.dout, self.out = (torch.randn(rows, hq, d, generator=gen).to(dtype).cuda() for _ in range(3))
        self.k, self.v = (torch.randn(kv_rows, hkv, d, generator=gen).to(dtype).cuda() for _ in range(2))
        self.lse = torch.randn(rows, hq, generator=gen).cuda()
        lens = [[n * ((i + 1) % 2) * (i < 2 * times) for i in range(batch)] for n in (rows, kv_rows)]
        self.cu = [prefix_sums(n).cuda() for n in lens] + [falling(batch, n, times).cuda() for n in (rows, kv_rows)]
        self.sound = [prefix_sums(x).cuda() for x in ([rows] + [0] * (batch - 1), [kv_rows] + [0] * (batch - 1))] * 2

    def nans(self):
        return [torch.full_like(x, float("nan")) for x in (self.q, self.k, self.v)]

    def run(self, call, need):
        """call(workspace): its outputs are zeros and its status is 1; then what lies behind."""
        held = torch.full((need + BEHIND,), 0xA5, dtype=torch.uint8, device="cuda")
        outputs = call(held[:need])
        assert ta.read_status(held[:need]) == 1
        assert not any(x.count_nonzero() for x in outputs)
        assert (held[need:] == 0xA5).all()


# ------------------------------------------------------------------ on the CPU
def test_tiles_of_sequences_side_by_side_fit():
    rng = np.random.default_rng(52)
    for _ in range(200):
        batch = int(rng.integers(1, 40))
        lens = [int(x) for x in 2 ** rng.uniform(0, 12, batch)]
        rows = sum(lens)
        assert sum((n + 127) // 128 for n in lens) <= room_for_tiles(batch, rows, rows)


def test_tiles_of_overlapping_sequences_need_not():
    """The offsets of the calls below."""
    assert falling(5, 9).tolist() == [0, 9, 0, 9, 0, 9]
    batch, rows = 19, 1300
    assert 10 * ((rows + 127) // 128) > room_for_tiles(batch, rows, 260)


def test_parts_of_sequences_side_by_side_fit():
    rng, cut = np.random.default_rng(53), 0
    for _ in range(400):
        batch, window, sinks = int(rng.integers(1, 12)), int(2 ** rng.uniform(0, 10)), int(rng.choice([1, 100, 129, 300, 5000]))
        lens = [int(x) for x in 2 ** rng.uniform(5, 15, batch)]
        edge = [2049, 2048 + 128, 4097, 6145]  # just past one, two, three parts
        lens = [edge[int(rng.integers(4))] if rng.random() < 0.5 else n for n in lens]
        keys = [max(1, n + int(rng.integers(-400, 400))) for n in lens]
        parts = sum(parts_of(n, m, window, sinks, low) for low in [bool(rng.integers(2))] for n, m in zip(lens, keys))
        cut += parts > 0
        assert parts <= room_for_parts(batch, sum(lens), sum(keys), window, sinks) or parts == 0
    assert cut > 200


FEW = dict(batch=60, rows=2200, kv_rows=128, times=4)  # whose tiles have room, and parts have not


def test_parts_of_overlapping_sequences_need_not():
    batch, rows, keys = FEW["batch"], FEW["rows"], FEW["kv_rows"]
    assert FEW["times"] * ((rows + 127) // 128) <= room_for_tiles(batch, rows, keys)
    assert FEW["times"] * parts_of(rows, keys, 64, 4, False) > room_for_parts(batch, rows, keys, 64, 4) > 0


# ------------------------------------------------------------------ on the GPU
@gpu
@pytest.mark.parametrize("mask", ["padding", "padding_causal", "padding_causal_bottom_right"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_packed_calls(d, mask):
    c = Overlap(d=d)

    def fwd(ws):
        out, lse = (torch.full_like(x, float("nan")) for x in (c.q, c.lse))
        return ta.fwd(c.q, c.k, c.v, *c.cu, 0.1, mask, out=out, lse=lse, workspace=ws)

    def bwd(ws, **kw):
        dq, dk, dv = c.nans()
        return ta.bwd(c.q, c.k, c.v, c.out, c.dout, c.lse, *c.cu, 0.1, mask, dq=dq, dk=dk, dv=dv, workspace=ws, **kw)
    c.run(fwd, ta.fwd_workspace_size(*c.sizes))
    c.run(bwd, ta.bwd_workspace_size(*c.sizes))
    if d <= 128:
        c.run(lambda ws: bwd(ws, fused=True), ta.bwd_fused_workspace_size(*c.sizes))
    # and the next call with the same workspace is none the worse
    ws = torch.empty(ta.bwd_workspace_size(*c.sizes), dtype=torch.uint8, device="cuda")
    bwd(ws)
    out, lse = ta.fwd(c.q, c.k, c.v, *c.sound, 0.1, mask)
    args = (c.q, c.k, c.v, out, c.dout, lse, *c.sound, 0.1, mask)
    again, want = ta.bwd(*args, workspace=ws), ta.bwd(*args)
    assert ta.read_status(ws) == 0 and all(torch.equal(a, b) for a, b in zip(again, want))


@gpu
def test_built_in_scratch():
    c = Overlap()
    dq, dk, dv = c.nans()
    got = ta.bwd_noalloc(c.q, c.k, c.v, c.out, c.dout, c.lse, *c.cu, 0.1, "padding", dq=dq, dk=dk, dv=dv)
    assert ta.read_status_noalloc() == 1 and not any(x.count_nonzero() for x in got)


@gpu
@pytest.mark.parametrize("window,sinks", [(64, 0), (64, 4), (300, 140)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_windowed_calls(d, window, sinks):
    """Sequences of 4096 queries over 128 keys: sweeps over sinks are cut, and have no room either."""
    c = Overlap(batch=21, rows=4096, kv_rows=128, d=d)

    def fwd(ws):
        out, lse = (torch.full_like(x, float("nan")) for x in (c.q, c.lse))
        return ta.window_fwd(c.q, c.k, c.v, *c.cu, 0.1, window, sinks, out=out, lse=lse, workspace=ws)

    def bwd(ws):
        dq, dk, dv = c.nans()
        return ta.window_bwd(c.q, c.k, c.v, c.out, c.dout, c.lse, *c.cu, 0.1, window, sinks, dq=dq, dk=dk, dv=dv, workspace=ws)
    c.run(fwd, ta.fwd_workspace_size(*c.sizes))
    c.run(bwd, ta.window_bwd_workspace_size(*c.sizes, window, sinks))


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_parts_of_cut_sweeps(d):
    """Offsets whose tiles have room, and whose parts of sweeps over sinks have not."""
    c = Overlap(d=d, **FEW)

    def bwd(ws):
        dq, dk, dv = c.nans()
        return ta.window_bwd(c.q, c.k, c.v, c.out, c.dout, c.lse, *c.cu, 0.1, 64, 4, dq=dq, dk=dk, dv=dv, workspace=ws)
    need = ta.window_bwd_workspace_size(*c.sizes, 64, 4)
    c.run(bwd, need)
    with ta.debug_build():
        c.run(bwd, need)


LOW = -2 ** 31


def _far_below(rows, kv_rows):
    """Three sequences of 20, none and 30 tokens. The offset between the first and the third lies so far
    below zero that the first one's span, as a 32-bit difference, looks long."""
    sound = [prefix_sums([0, 0, 30])] * 2 + [torch.tensor([0, 30, 30, n], dtype=torch.int32) for n in (rows, kv_rows)]
    bad = [prefix_sums([20, 0, 30])] * 2 + [torch.tensor([5, LOW, 30, n], dtype=torch.int32) for n in (rows, kv_rows)]
    return [[x.cuda() for x in cu] for cu in (sound, bad)]


def test_a_difference_that_wraps():
    """What the tests of such offsets relies on: in 32 bits the span from 5 to -2^31 is long."""
    assert np.subtract(np.int32(LOW), np.int32(5), dtype=np.int32) == 2 ** 31 - 5


@gpu
@pytest.mark.parametrize("window", [0, 12])
@pytest.mark.parametrize("d", [64, 256])
def test_offsets_far_below_zero(d, window):
    """They leave the sequence beside them empty and the others as they are."""
    c = Overlap(rows=70, kv_rows=66, d=d)
    sound, bad = _far_below(70, 66)
    head = (c.q, c.k, c.v)
    size = (3, 70, 66, 4, 2, d)

    def both(cu):
        wf = torch.empty(ta.fwd_workspace_size(*size), dtype=torch.uint8, device="cuda")
        out, lse = torch.full_like(c.q, float("nan")), torch.full_like(c.lse, float("nan"))
        g = dict(zip(("dq", "dk", "dv"), c.nans()))
        if window:
            wb = torch.empty(ta.window_bwd_workspace_size(*size, window, 2), dtype=torch.uint8, device="cuda")
            ta.window_fwd(*head, *cu, 0.1, window, 2, out=out, lse=lse, workspace=wf)
            ta.window_bwd(*head, out, c.dout, lse, *cu, 0.1, window, 2, workspace=wb, **g)
        else:
            wb = torch.empty(ta.bwd_workspace_size(*size), dtype=torch.uint8, device="cuda")
            ta.fwd(*head, *cu, 0.1, "padding_causal", out=out, lse=lse, workspace=wf)
            ta.bwd(*head, out, c.dout, lse, *cu, 0.1, "padding_causal", workspace=wb, **g)
        return (out, lse, *g.values()), ta.read_status(wf), ta.read_status(wb)
    want, *clean = both(sound)
    got, *status = both(bad)
    assert clean == [0, 0] and status == [1, 1]
    assert all(torch.equal(a, b) for a, b in zip(want, got))
