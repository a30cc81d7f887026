"""Shared-prefix attention and rotations at sizes where index arithmetic runs out of bits."""

import ctypes
import math

import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from prefix_common import ROUNDOFF, TINY, prefix_sums

gpu = pytest.mark.gpu


@gpu
def test_gradients_of_a_cache_of_many_keys():
    """64 heads on one kv head and 34 million own keys behind the lower-right triangle: a key's
    distance from the first query, times the 64 packed heads, is past 2^31. lse and out are
    inputs of the backward, so dk and dv of some keys follow from the formula at any values of
    theirs: P = exp(scale q k - lse), dS = P (dO v - rowsum(dO out)).

    The bound: P and dS are rounded once to 16 bits (u of each term) and the result once (u), u
    for fp32 (2^-20 of the terms of scores of at most a few units, of dO v and of rowsum)."""
    hq, d, n, m, prefix = 64, 8, 4, 34_000_000, 10
    dtype, scale = torch.bfloat16, 1.0 / math.sqrt(8)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)
    q, out, dout = rand(n, hq, d), rand(n, hq, d), rand(n, hq, d)
    k, v, kp, vp = rand(m, 1, d), rand(m, 1, d), rand(prefix, 1, d), rand(prefix, 1, d)
    lse = torch.randn((n, hq), generator=gen, device="cuda") * 0.5
    cu_q, cu_k = prefix_sums([n]).cuda(), prefix_sums([m]).cuda()
    ws = torch.empty(ta.prefix_bwd_workspace_size(1, n, m, prefix, hq, 1, d), dtype=torch.uint8, device="cuda")
    dq, dk, dv, dkp, dvp = ta.prefix_bwd(q, k, v, kp, vp, out, dout, lse, cu_q, cu_k, cu_q, cu_k, scale,
                                         "padding_causal_bottom_right", workspace=ws)
    assert ta.read_status(ws) == 0
    edge = m - n - 2 ** 31 // 64
    keys = torch.cat([torch.arange(a, a + 300) for a in (0, edge - 150, m // 2, m - 300)]).cuda()
    Q, G, O = (x.double().flatten(0, 1) for x in (q, dout, out))
    token = torch.arange(n, device="cuda").repeat_interleave(hq)
    for K, V, gk, gv, see in ((k[keys, 0], v[keys, 0], dk[keys, 0], dv[keys, 0], keys[None] <= token[:, None] + m - n),
                              (kp[:, 0], vp[:, 0], dkp[:, 0], dvp[:, 0], torch.ones(n * hq, prefix, dtype=torch.bool, device="cuda"))):
        K, V = K.double(), V.double()
        P = torch.where(see, torch.exp(scale * Q @ K.T - lse.double().flatten()[:, None]), 0.0)
        D = (G * O).sum(1, keepdim=True)
        dS = P * (G @ V.T - D)
        far = 2.0 ** -20 * P * (G.abs() @ V.abs().T + (G * O).abs().sum(1, keepdim=True))
        u = ROUNDOFF[dtype]
        for got, ref, size in ((gv, P.T @ G, P.T @ G.abs()), (gk, scale * dS.T @ Q, scale * (dS.abs() + far / u).T @ Q.abs())):
            over = ((got.double() - ref).abs() - 2 * u * (size + ref.abs()) - TINY[dtype]).max().item()
            assert over <= 0, over


def _bwd_code(batch, total_q, total_kv, rows, hq, hkv, d):
    """What the backward answers, with placeholder pointers and no launch, for a size."""
    P, cu = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)
    return ta.library().te_attn_prefix_bwd_thd(*[P] * 13, cu, cu, cu, cu, None, batch, total_q, total_kv, rows, hq, hkv, d,
                                               0.1, 1, 1, P, ctypes.c_size_t(1 << 60), None)


def test_more_steps_than_an_item_can_tell():
    """A dK/dV item hands its number of steps over in 24 bits. Cutting the prefix's sweep does
    not shorten the items of a sequence's own keys, which take as many steps if it holds all
    queries: 16,000,001 heads (an odd group, a head at a time) of two row tiles are refused."""
    size = (2, 129, 64, 32, 16_000_001, 1, 8)
    assert ta.prefix_bwd_workspace_size(*size) == 0
    assert _bwd_code(*size) == -2
    assert ta.prefix_bwd_workspace_size(2, 129, 64, 32, 8_000_001, 1, 8) > 0


def test_sizes_within_a_tile_of_2_to_the_31():
    """Rounding a length up to whole tiles must not pass 2^31: sizes that close are refused, by
    the sizes' functions and by the calls; those a tile below are not."""
    top = 2 ** 31 - 1
    for size in ((1, 64, top, 32, 1, 1, 8), (1, 64, top - 255, 32, 1, 1, 8), (1, 64, 64, top, 1, 1, 8),
                 (1, top, 64, 32, 1, 1, 8), (1, top // 3, 64, 32, 3, 1, 8)):
        assert ta.prefix_fwd_workspace_size(*size) == 0 and ta.prefix_bwd_workspace_size(*size) == 0, size
        assert _bwd_code(*size) == -2, size
        P, cu = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)
        assert ta.library().te_attn_prefix_fwd_thd(*[P] * 7, cu, cu, cu, cu, None, *size, 0.1, 1, 1, P,
                                                   ctypes.c_size_t(1 << 60), None) == -2, size
    assert ta.prefix_fwd_workspace_size(1, 64, top - 256, top - 256, 1, 1, 8) > 0
    assert ta.prefix_bwd_workspace_size(1, 64, top - 256, top - 256, 1, 1, 8) > 0
    P = ctypes.c_void_p(1 << 20)
    for rows in (top, top - 255):  # a rotation's blocks take up to four tokens
        assert ta.library().te_attn_rope_thd(P, P, P, P, P, 4, P, P, None, 1, rows, 1, 1, 8, 8, 8, 8, 8, 0, 1.0, 0, 1, None) == -1


def test_more_frequencies_than_a_head_has_pairs():
    """Any number of frequencies above d / 2 is refused, those whose double passes 2^31 too."""
    P = ctypes.c_void_p(1 << 20)
    for n in (33, 1 << 30, (1 << 31) - 1):
        assert ta.library().te_attn_rope_thd(P, P, P, P, P, n, P, P, None, 1, 4, 1, 1, 64, 64, 64, 64, 64, 0, 1.0, 0, 1, None) == -1
