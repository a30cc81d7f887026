"""Shared-prefix attention over many sequences, short and long ones mixed: the scheduler's
records of a sequence are then read by other warps than the one that wrote them, and its
loops over sequences take several passes."""

import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from prefix_common import prefix_check
from test_prefix import ALL, BR, FWD, TL, Case, _same

gpu = pytest.mark.gpu


def _lengths(batch, group, longest):
    """Query lengths of which about half come to more than 128 rows of a kv head (with tile
    counts of 1 to a few) and the others to fewer, some of them none; own keys from none to
    more than the queries."""
    edge = 128 // group
    lq = []
    for i in range(batch):
        r = (i * 37 + i * i * 11) % 101
        lq.append(edge + 1 + r * (longest - edge - 1) // 100 if (i * 7919 >> 3) % 2 else (r % (edge + 1)) * (i % 3) // 2)
    lk = [n + (13 * i) % 29 if i % 4 else (5 * i) % 23 for i, n in enumerate(lq)]
    return lq, lk


@gpu
@pytest.mark.parametrize("batch,d,hq,hkv,dtype,mask,longest", [(300, 128, 8, 2, torch.bfloat16, BR, 190),
                                                               (420, 64, 6, 1, torch.float16, TL, 120),
                                                               (270, 256, 8, 1, torch.bfloat16, BR, 60),
                                                               (1100, 64, 4, 1, torch.bfloat16, BR, 70),
                                                               (1060, 136, 4, 2, torch.float16, TL, 90)])
def test_short_and_long_sequences(batch, d, hq, hkv, dtype, mask, longest):
    """Against the definition, forward and backward; then the same bits on workspaces that a call
    with other lengths left behind and on poisoned ones."""
    lq, lk = _lengths(batch, hq // hkv, longest)
    assert sum(n * hq // hkv > 128 for n in lq) > 100 and sum(0 < n * hq // hkv <= 128 for n in lq) > 40
    c = Case(batch + d, lq, lk, 77, hq, hkv, d, dtype, mask, slot_q=1, slot_k=4)
    other = Case(batch, lq[::-1], lk[::-1], 77, hq, hkv, d, dtype, mask, slot_q=1, slot_k=4).dev()
    assert other.q.shape == c.q.shape and other.k.shape == c.k.shape
    sizes = (batch, c.q.shape[0], c.k.shape[0], 77, hq, hkv, d)
    ws, wsb = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in
               (ta.prefix_fwd_workspace_size(*sizes), ta.prefix_bwd_workspace_size(*sizes)))
    out, lse = c.fwd(workspace=ws)
    first = [out, lse, *c.bwd(out, lse, workspace=wsb)]
    assert ta.read_status(ws) == 0 and ta.read_status(wsb) == 0
    ref = c.plain()
    prefix_check({"out": out, "lse": lse, **dict(zip(ALL, first[2:]))}, ref, FWD + ALL, dtype)
    for left in ("other", 0xff, 0x00, 0x7f):
        if left == "other":
            o, l = other.fwd(workspace=ws)
            other.bwd(o, l, workspace=wsb)
        else:
            ws.fill_(left)
            wsb.fill_(left)
        o, l = c.fwd(workspace=ws)
        again = [o, l, *c.bwd(o, l, workspace=wsb)]
        assert ta.read_status(ws) == 0 and ta.read_status(wsb) == 0
        assert _same(first, again)
