"""Rotary positions against their definition in 64 bits, forward, backward and refusals."""

import ctypes
import math

import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from prefix_common import prefix_sums, rope_check, rope_plain

gpu = pytest.mark.gpu


def test_plain_form_is_a_complex_product():
    """The tests' reference turns pairs as complex numbers, and the inverse undoes it."""
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(5, 2, 16, generator=gen, dtype=torch.float64)
    w, _ = ta.rope_frequencies(8, device="cpu")
    y, _ = rope_plain(x, w, [5], [0], [7], False, 1.0)
    z = torch.complex(x[..., :4], x[..., 4:8]) * torch.exp(1j * (7 + torch.arange(5))[:, None, None] * w)
    assert torch.allclose(y[..., :8], torch.cat((z.real, z.imag), -1)) and torch.equal(y[..., 8:], x[..., 8:])
    back, _ = rope_plain(y, w, [5], [0], [7], False, 1.0, inverse=True)
    assert torch.allclose(back, x)


def test_frequencies():
    """Unscaled, linear, ntk and yarn frequencies from their definitions."""
    n, base, f = 64, 10000.0, 8.0
    w, m = ta.rope_frequencies(n, device="cpu")
    assert w.dtype == torch.float64 and m == 1.0
    assert w[0] == 1.0 and math.isclose(w[5], base ** (-10 / n), rel_tol=1e-14)
    lin, m = ta.rope_frequencies(n, scaling="linear", factor=f, device="cpu")
    assert torch.allclose(lin, w / f, rtol=1e-15) and m == 1.0
    ntk, _ = ta.rope_frequencies(n, scaling="ntk", factor=f, device="cpu")
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], w[-1] / f, rel_tol=1e-12)
    yarn, m = ta.rope_frequencies(n, scaling="yarn", factor=f, original_length=4096, device="cpu")
    assert yarn[0] == w[0] and math.isclose(yarn[-1], w[-1] / f, rel_tol=1e-12)
    assert math.isclose(m, 0.1 * math.log(f) + 1) and bool((yarn <= w).all()) and bool((yarn >= w / f).all())
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, scaling="other"), dict(rot_dim=8, factor=0.5)):
        with pytest.raises(ValueError):
            ta.rope_frequencies(**bad, device="cpu")


def test_refusals_launch_nothing():
    """Bad arguments return their code before any launch (placeholder pointers)."""
    lib = ta.library()
    P, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)

    def call(q=P, k=P, qo=P, ko=P, w=P, n=16, cu=P, pad=P, start=None, batch=2, total=64, hq=4, hkv=2, d=64,
             st=256, m=1.0, dtype=1):
        return lib.te_attn_rope_thd(q, k, qo, ko, w, n, cu, pad, start, batch, total, hq, hkv, d, st, 64, st,
                                    64, 0, m, 0, dtype, None)
    assert call(d=12) == -2 and call(d=264) == -2 and call(dtype=3) == -2
    assert call(n=0) == -1 and call(n=33) == -1
    assert call(batch=0) == -1 and call(total=-1) == -1 and call(hq=0) == -1 and call(hkv=-1) == -1
    assert call(w=None) == -1 and call(cu=None) == -1 and call(pad=None) == -1
    assert call(q=None) == -1 and call(ko=None) == -1
    assert call(q=odd) == -1 and call(w=ctypes.c_void_p((1 << 20) + 4)) == -1
    assert call(st=-8) == -1 and call(st=(1 << 31) + 8) == -1
    assert call(m=float("nan")) == -1 and call(m=float("inf")) == -1
    assert lib.te_attn_last_error()
    assert call(total=0) == 0  # nothing to do, nothing launched
    assert lib.te_attn_rope_sbhd(P, P, P, P, P, 16, P, None, 2, 1 << 30, 4, 2, 64, 8, 8, 8, 8, 0, 1.0, 0, 1, None) == -1
    assert lib.te_attn_rope_sbhd(P, P, P, P, P, 16, P, None, 0, 8, 4, 2, 64, 8, 8, 8, 8, 0, 1.0, 0, 1, None) == -1
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    w, _ = ta.rope_frequencies(64, device="cpu")
    cu = prefix_sums([4])
    with pytest.raises(ValueError):
        ta.rope(q, None, w, cu, cu)
    with pytest.raises(ValueError):
        ta.rotary_positions(q, None, w)
    with pytest.raises(NotImplementedError):
        ta.rotary_positions(q, None, w, cu, qkv_format="hbsd")


def _packed(seed, lengths, slots, hq, hkv, d, dtype, extra=3):
    """Strided q and k (slices of a fused tensor) with NaN in every row that is no token."""
    gen = torch.Generator().manual_seed(seed)
    offs = [0]
    for s in slots:
        offs.append(offs[-1] + s)
    x = torch.randn(offs[-1] + extra, hq + 2 * hkv, d, generator=gen).to(dtype)
    keep = torch.zeros(x.shape[0], dtype=torch.bool)
    for n, o in zip(lengths, offs):
        keep[o:o + n] = True
    x[~keep] = float("nan")
    return x, offs, keep


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,dtype", [(128, 128, torch.bfloat16), (64, 32, torch.float16), (80, 20, torch.bfloat16),
                                         (48, 24, torch.float16), (8, 2, torch.bfloat16), (256, 256, torch.float16),
                                         (40, 6, torch.float16)])
def test_packed_matches_definition(d, rot, dtype, interleaved):
    """Ragged lengths (0 and 1 among them), far starts, strided inputs, NaN in pad rows,
    forward and inverse; pad rows and the tail come out as zeros."""
    lengths, slots = [5, 0, 1, 33, 2], [8, 3, 1, 33, 7]
    hq, hkv = 6, 2
    x, offs, keep = _packed(d + rot, lengths, slots, hq, hkv, d, dtype)
    w, _ = ta.rope_frequencies(rot, device="cpu")
    starts = [0, 5, 1000003, 130000, 77]
    cu, pad = prefix_sums(lengths).cuda(), prefix_sums(slots).cuda()
    st = torch.tensor(starts, dtype=torch.int32).cuda()
    xd = x.cuda()
    for inverse in (False, True):
        qo, ko = ta.rope(xd[:, :hq], xd[:, hq:hq + hkv], w.cuda(), cu, pad, st, interleaved, 1.25, inverse)
        for got, part in ((qo, x[:, :hq]), (ko, x[:, hq:hq + hkv])):
            ref, size = rope_plain(part, w, lengths, offs, starts, interleaved, 1.25, inverse)
            assert got.is_contiguous() and torch.equal(got.cpu()[~keep], torch.zeros_like(part[~keep]))
            rope_check(got, ref, size, f"inverse {inverse}")


@gpu
@pytest.mark.parametrize("shift,step", [(1, 1), (2, 3), (4, 4), (0, 8)])
def test_unaligned_strides(shift, step):
    """Inputs whose base or strides allow only narrower accesses give the same bits."""
    T, h, d = 9, 3, 64
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(T, h, d, generator=gen).to(torch.bfloat16).cuda()
    w, _ = ta.rope_frequencies(d)
    cu = prefix_sums([T]).cuda()
    ref, _ = ta.rope(x, None, w, cu, cu)
    buf = torch.zeros(T * (h * (d + step) + step) + shift + 64, dtype=torch.bfloat16, device="cuda")
    view = buf.as_strided((T, h, d), (h * (d + step) + step, d + step, 1), shift)
    view.copy_(x)
    got, none = ta.rope(view, None, w, cu, cu)
    assert none is None and torch.equal(got.view(torch.int16), ref.view(torch.int16))


@gpu
def test_in_place_and_expanded():
    """An output may be its input; a zero stride (one row for all) is read as such."""
    T, h, d = 40, 4, 128
    x = torch.randn(T, h, d, generator=torch.Generator().manual_seed(5)).to(torch.float16).cuda()
    w, _ = ta.rope_frequencies(d)
    cu = prefix_sums([T]).cuda()
    ref, _ = ta.rope(x, None, w, cu, cu)
    same = x.clone()
    out, _ = ta.rope(same, None, w, cu, cu, q_out=same)
    assert out.data_ptr() == same.data_ptr() and torch.equal(out, ref)
    one, _ = ta.rope(x[:1].expand(T, h, d), None, w, cu, cu)
    full, _ = ta.rope(x[:1].expand(T, h, d).contiguous(), None, w, cu, cu)
    assert torch.equal(one, full)


@gpu
def test_bad_lengths_give_zero_rows():
    """A sequence whose real length or slot does not fit is treated as empty."""
    x = torch.randn(16, 2, 64, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    w, _ = ta.rope_frequencies(64)
    cu, pad = (torch.tensor(c, dtype=torch.int32).cuda() for c in ([0, 4, 12, 14], [0, 4, 8, 40]))
    out, _ = ta.rope(x, None, w, cu, pad)
    ref, size = rope_plain(x, w, [4], [0], [0], False, 1.0)
    rope_check(out, ref, size)
    assert torch.equal(out[4:], torch.zeros_like(out[4:]))


@gpu
@pytest.mark.parametrize("fmt", ["thd", "bshd", "sbhd"])
def test_autograd_and_layouts(fmt):
    """Values and gradients through autograd in the three layouts; sum() hands back an
    expanded gradient."""
    B, S, hq, hkv, d = 3, 11, 4, 2, 64
    gen = torch.Generator().manual_seed(8)
    lengths = [11, 4, 7]
    starts = torch.tensor([3, 0, 500], dtype=torch.int32)
    w, m = ta.rope_frequencies(32, scaling="yarn", factor=4.0)
    q, k = (torch.randn(B, S, h, d, generator=gen).to(torch.bfloat16) for h in (hq, hkv))
    gq, gk = (torch.randn(B, S, h, d, generator=gen).to(torch.bfloat16) for h in (hq, hkv))
    cu, pad = prefix_sums(lengths), prefix_sums([S] * B)

    def lay(x):
        return x.transpose(0, 1).contiguous() if fmt == "sbhd" else x if fmt == "bshd" else x.flatten(0, 1)

    def unlay(x):
        x = x.detach().cpu()
        return (x.transpose(0, 1) if fmt == "sbhd" else x.view(B, S, x.shape[-2], d)).reshape(B * S, x.shape[-2], d)
    a, b = (lay(x).cuda().requires_grad_() for x in (q, k))
    extra = {"cu_seqlens_padded": pad.cuda()} if fmt == "thd" else {}
    qo, ko = ta.rotary_positions(a, b, w, cu.cuda(), start_positions=starts.cuda(), mscale=m, qkv_format=fmt, **extra)
    torch.autograd.backward((qo, ko), (lay(gq).cuda(), lay(gk).cuda()))
    offs = [0, S, 2 * S]
    for got, x, inverse in ((qo, q, False), (ko, k, False), (a.grad, gq, True), (b.grad, gk, True)):
        ref, size = rope_plain(x.flatten(0, 1), w, lengths, offs, starts.tolist(), False, m, inverse)
        rope_check(unlay(got), ref, size)
    a.grad = None
    qo, _ = ta.rotary_positions(a, b, w, cu.cuda(), start_positions=starts.cuda(), mscale=m, qkv_format=fmt, **extra)
    qo.sum().backward()
    ref, size = rope_plain(torch.ones(B * S, hq, d), w, lengths, offs, starts.tolist(), False, m, True)
    rope_check(unlay(a.grad), ref, size)


@gpu
def test_gradient_against_differences():
    """The gradient against central differences of the op itself, on the linear functional
    <g, rope(x)>: the op is linear, so a difference over a unit step is exact up to rounding."""
    gen = torch.Generator().manual_seed(9)
    x, g = (torch.randn(6, 1, 16, generator=gen).to(torch.float16).cuda() for _ in range(2))
    w, _ = ta.rope_frequencies(8)
    cu = prefix_sums([6]).cuda()
    grad, _ = ta.rope(g, None, w, cu, cu, inverse=True)
    for t, c in ((0, 0), (3, 1), (5, 6), (2, 12)):
        e = torch.zeros_like(x)
        e[t, 0, c] = 1.0
        plus, minus = (ta.rope(x.float().add(s * e.float()).half(), None, w, cu, cu)[0] for s in (1, -1))
        num = ((plus.double() - minus.double()) * g.double()).sum().item() / 2
        # four roundings of 2^-11 of values up to 5 (|x| + 1), times |g| of a pair
        tol = 4 * 2.0 ** -11 * 5 * g.double().abs().max().item()
        assert abs(num - grad[t, 0, c].item()) <= tol


@gpu
def test_captured_replay_and_side_stream():
    """A replayed graph gives an eager call's bits on new inputs; a call on another stream too."""
    gen = torch.Generator().manual_seed(10)
    q, k = (torch.randn(70, h, 128, generator=gen).to(torch.bfloat16).cuda() for h in (8, 2))
    w, _ = ta.rope_frequencies(128)
    cu, pad = prefix_sums([30, 20]).cuda(), prefix_sums([32, 32]).cuda()
    outs = ta.rope(q, k, w, cu, pad)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ta.rope(q, k, w, cu, pad, q_out=outs[0], k_out=outs[1])
    q.copy_(torch.randn(q.shape, generator=gen))
    g.replay()
    ref = ta.rope(q, k, w, cu, pad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = ta.rope(q, k, w, cu, pad)
    torch.cuda.synchronize()
    for a, b, c in zip(outs, ref, other):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(b.view(torch.int16), c.view(torch.int16))


@gpu
def test_arguments_that_do_not_fit_are_refused():
    """Shapes, types and devices that do not go together, before any launch."""
    x = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    w, _ = ta.rope_frequencies(64)
    cu = prefix_sums([8]).cuda()

    def call(q=x, k=None, w=w, cu=cu, pad=cu, **kw):
        with pytest.raises((ValueError, RuntimeError)):
            ta.rope(q, k, w, cu, pad, **kw)
    call(q=x.float())
    call(k=x.half())
    call(k=x[:-1])
    call(k=x[..., :32])
    call(q=x.transpose(1, 2))
    call(q=x[0])
    call(w=w.float())
    call(w=w.cpu())
    call(w=torch.cat((w, w)))
    call(cu=cu.long())
    call(pad=cu[:-1])
    call(start_positions=cu)
    call(q_out=x[:-1])
    call(k_out=x)
    call(mscale=float("nan"))
    call(q=torch.zeros(1, 4097, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        ta.rope_sbhd(x.view(4, 2, 2, 64), None, w, prefix_sums([4]).cuda())


@gpu
def test_nothing_to_turn():
    """No rows, and rows without a sequence of any length."""
    w, _ = ta.rope_frequencies(64)
    cu = prefix_sums([0, 0]).cuda()
    out, _ = ta.rope(torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda"), None, w, cu, cu)
    assert out.shape == (0, 2, 64)
    x = torch.full((5, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    out, k = ta.rope(x, x, w, cu, cu)
    assert torch.equal(out, torch.zeros_like(x)) and torch.equal(k, torch.zeros_like(x))


@gpu
def test_given_outputs_and_streams():
    """Outputs that the caller gives come back as the same objects, also on another stream."""
    gen = torch.Generator().manual_seed(12)
    q, k = (torch.randn(20, h, 64, generator=gen).to(torch.float16).cuda() for h in (4, 2))
    w, _ = ta.rope_frequencies(64)
    cu = prefix_sums([20]).cuda()
    ref = ta.rope(q, k, w, cu, cu)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    got = ta.rope(q, k, w, cu, cu, None, False, 1.0, False, qo, ko)
    assert got[0] is qo and got[1] is ko
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = ta.rope(q, k, w, cu, cu, stream=side.cuda_stream)
    side.synchronize()
    for a, b, c in zip(ref, got, other):
        assert torch.equal(a, b) and torch.equal(a, c)
    with pytest.raises(ValueError):
        ta.rope(q, None, w, cu, None)
