"""Kernel timing of shared-prefix calls: what is recorded, and that it changes no result."""

import ctypes

import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from test_prefix import BR, Case, _same

gpu = pytest.mark.gpu
SCHEDULE, FWD, DELTA, DKDV, DQ, KERNELS = 0, 1, 3, 4, 5, 9


@gpu
def test_recorded_launches():
    """Events between the launches of a call, which otherwise start before the one ahead of them
    has ended: the same bits; two launches forward beside the scheduler, and the sum of the
    prefix's parts counted with dK/dV."""
    lib = ta.library()
    c = Case(41, [300, 1, 77, 40], [300, 9, 77, 40], 200, 8, 2, 64, torch.bfloat16, BR).dev()
    sizes = (4, c.q.shape[0], c.k.shape[0], 200, 8, 2, 64)
    ws, wsb = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in
               (ta.prefix_fwd_workspace_size(*sizes), ta.prefix_bwd_workspace_size(*sizes)))
    out, lse = c.fwd(workspace=ws)
    first = [out, lse, *c.bwd(out, lse, workspace=wsb)]
    torch.cuda.synchronize()
    ms, n = (ctypes.c_double * KERNELS)(), (ctypes.c_int * KERNELS)()
    assert lib.te_attn_profile_enable(1) == 0
    try:
        for _ in range(5):
            o, l = c.fwd(workspace=ws)
            assert _same(first, [o, l, *c.bwd(o, l, workspace=wsb)])
        assert lib.te_attn_profile_read(ms, n) == 0
    finally:
        assert lib.te_attn_profile_enable(0) == 0
    count = list(n)
    assert count[SCHEDULE] == 10 and count[FWD] == 10 and count[DELTA] == 5 and count[DQ] == 5 and count[DKDV] in (5, 10)
    assert sum(count) == 30 + count[DKDV] and all((t > 0) == (k > 0) for t, k in zip(ms, count))
