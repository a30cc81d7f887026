"""What autograd hands to the backward of shared-prefix attention."""

import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from test_prefix import TL, Case

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("lead", [1, 3, 8])
def test_gradient_that_starts_anywhere(lead):
    """The gradient of a flattened, joined output is a slice of the joined one's, adjacent but
    not on a 16-byte boundary: the same bits as from a gradient of its own."""
    c = Case(6, [9, 1, 30], [9, 1, 30], 40, 4, 2, 64, torch.bfloat16, TL).dev()
    leaves = [x.clone().requires_grad_() for x in c.on]
    out = ta.shared_prefix_attention(*leaves, *c.cu_on)
    ref = torch.autograd.grad(out, leaves, c.dout_on.view(out.shape), retain_graph=True)
    joined = torch.cat((torch.zeros(lead, dtype=out.dtype, device="cuda"), out.flatten()))
    g = torch.cat((torch.zeros(lead, dtype=out.dtype, device="cuda"), c.dout_on.flatten()))
    assert all(torch.equal(a, b) for a, b in zip(ref, torch.autograd.grad(joined, leaves, g)))
