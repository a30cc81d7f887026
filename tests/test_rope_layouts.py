"""Rotary positions on tensors with axes of one or no elements, whose strides mean nothing."""

import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from prefix_common import prefix_sums, rope_check, rope_plain

gpu = pytest.mark.gpu


def _bits(x):
    return x.contiguous().view(torch.int16)


@gpu
def test_sequence_major_batch_of_one():
    """[1, S, h, d] transposed to [S, 1, h, d]: torch calls that contiguous whatever the stride
    of the batch is. Values and gradients, also from a gradient laid out so."""
    S, h, d = 13, 4, 64
    gen = torch.Generator().manual_seed(1)
    w, m = ta.rope_frequencies(d)
    cu = prefix_sums([11]).cuda()
    x, g = (torch.randn(1, S, h, d, generator=gen).to(torch.bfloat16) for _ in range(2))
    ref, size = rope_plain(x[0], w, [11], [0], [0], False, m)
    back, back_size = rope_plain(g[0], w, [11], [0], [0], False, m, True)
    slice_of = torch.cat((x, x), 2).cuda()[:, :, h:]  # of a fused projection
    for q in (x.cuda().transpose(0, 1), slice_of.transpose(0, 1), x.cuda().as_strided((S, 1, h, d), (h * d, 8, d, 1))):
        assert q.shape == (S, 1, h, d)
        out, k = ta.rope_sbhd(q, q, w, cu, mscale=m)
        assert out.is_contiguous() and torch.equal(_bits(out), _bits(k))
        rope_check(out[:, 0], ref, size)
        leaf = q.detach().requires_grad_()
        y, _ = ta.rotary_positions(leaf, None, w, cu, mscale=m, qkv_format="sbhd")
        y.backward(g.cuda().transpose(0, 1))
        rope_check(leaf.grad[:, 0], back, back_size)


@gpu
def test_strides_of_axes_of_one():
    """One token, one head: a stride that nothing is reached by may have any value."""
    d = 64
    gen = torch.Generator().manual_seed(2)
    w, _ = ta.rope_frequencies(d)
    cu = prefix_sums([1]).cuda()
    start = torch.tensor([7], dtype=torch.int32).cuda()
    x = torch.randn(1, 1, d, generator=gen).to(torch.float16).cuda()
    ref, _ = ta.rope(x, None, w, cu, cu, start)
    for strides in ((1 << 40, d, 1), (d, 1 << 40, 1), (3, 5, 1)):
        got, k = ta.rope(x.as_strided((1, 1, d), strides), x.as_strided((1, 1, d), strides), w, cu, cu, start)
        assert torch.equal(_bits(got), _bits(ref)) and torch.equal(_bits(k), _bits(ref))


@gpu
@pytest.mark.parametrize("fmt,shape", [("bshd", (2, 0, 4, 64)), ("sbhd", (0, 2, 4, 64))])
def test_layouts_without_a_token(fmt, shape):
    """No token in any sequence: empty results and gradients, with lengths given or not."""
    w, _ = ta.rope_frequencies(64)
    x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    for cu in (None, prefix_sums([0, 0]).cuda()):
        q, k = ta.rotary_positions(x, x, w, cu, qkv_format=fmt)
        assert q.shape == k.shape == shape
        assert torch.autograd.grad(q, x, torch.zeros_like(q))[0].shape == shape
