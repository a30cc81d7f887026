"""Gradients of gradients: those of the rotation are rotations, those of shared-prefix
attention are refused instead of left out."""

import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from prefix_common import prefix_sums
from test_prefix import TL, Case

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("fmt", ["thd", "bshd", "sbhd"])
def test_rotation(fmt):
    """<g, rope(x)> has the gradient rope^-1(g) by x, whose gradient by g along r is rope(r); a
    penalty on the gradient reaches what the gradient came from."""
    B, S, h, d = 2, 9, 4, 64
    gen = torch.Generator().manual_seed(3)
    w, m = ta.rope_frequencies(32, scaling="yarn", factor=4.0)
    x, y, g, r = (torch.randn(B, S, h, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(4))
    if fmt == "thd":
        x, y, g, r = (t.flatten(0, 1) for t in (x, y, g, r))
    elif fmt == "sbhd":
        x, y, g, r = (t.transpose(0, 1).contiguous() for t in (x, y, g, r))
    cu = prefix_sums([S, 5]).cuda()
    kw = dict(mscale=m, qkv_format=fmt, **({"cu_seqlens_padded": prefix_sums([S, S]).cuda()} if fmt == "thd" else {}))
    x, g = x.requires_grad_(), g.requires_grad_()
    for k in (None, y.requires_grad_()):
        q, k2 = ta.rotary_positions(x, k, w, cu, **kw)
        gx, = torch.autograd.grad(q, x, g, create_graph=True)
        plain, = torch.autograd.grad(ta.rotary_positions(x, k, w, cu, **kw)[0], x, g)
        assert gx.requires_grad and torch.equal(gx.detach(), plain)
        gg, = torch.autograd.grad(gx, g, r, retain_graph=True)
        assert torch.equal(gg, ta.rotary_positions(r, None, w, cu, **kw)[0])
        penalty, = torch.autograd.grad((gx.float() ** 2).sum(), g)
        assert torch.equal(penalty, ta.rotary_positions((2 * gx.detach().float()).to(gx.dtype), None, w, cu, **kw)[0])


@gpu
def test_shared_prefix_attention():
    """The first gradients are there, with a graph wanted or not, and the same; going through them
    again raises, also where other terms of the loss could hide that nothing came of it."""
    c = Case(5, [9, 1, 30], [9, 1, 30], 40, 4, 2, 64, torch.bfloat16, TL).dev()
    leaves = [x.clone().requires_grad_() for x in c.on]

    def grads(**kw):
        out = ta.shared_prefix_attention(*leaves, *c.cu_on)
        return torch.autograd.grad(out, leaves, c.dout_on.view(out.shape), **kw)
    first, again = grads(), grads(create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    for g, x in zip(again, leaves):
        with pytest.raises(RuntimeError, match="second derivatives"):
            ((g.float() ** 2).sum() + x.float().sum()).backward(retain_graph=True)
