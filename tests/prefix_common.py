"""Plain 64-bit forms of the rotary and shared-prefix operators, for their tests, with
bounds on how far 16-bit results may lie from them."""

from __future__ import annotations

import math

import numpy as np
import torch

ROUNDOFF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
# half the spacing of subnormals: the absolute error of rounding a tiny value
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def prefix_sums(lengths):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32)


def rope_plain(x, inv_freq, lengths, offsets, starts, interleaved, mscale, inverse=False):
    """(rotated x, |x1| + |x2| of each element's pair) in float64 for packed x [T, h, d]."""
    x = x.detach().cpu().double()
    w = inv_freq.detach().cpu().double()
    half = w.numel()
    y, size = torch.zeros_like(x), torch.zeros_like(x)
    for n, off, s in zip(lengths, offsets, starts):
        for i in range(n):
            a = (s + i) * w * (-1.0 if inverse else 1.0)
            cos, sin = a.cos() * mscale, a.sin() * mscale
            row = x[off + i]
            one = torch.arange(half) * 2 if interleaved else torch.arange(half)
            two = one + 1 if interleaved else one + half
            y[off + i] = row
            y[off + i][:, one] = row[:, one] * cos - row[:, two] * sin
            y[off + i][:, two] = row[:, two] * cos + row[:, one] * sin
            size[off + i][:, one] = size[off + i][:, two] = row[:, one].abs() + row[:, two].abs()
    return y, size * abs(mscale)


def rope_check(got, ref, size, what=""):
    """One rounding to 16 bits, plus fp32's: sincospif errs by at most 2 ulp (2^-22 at 1), the
    angle's rounding moves it by at most pi 2^-24 relative to half a turn, and the products and
    their sum add 3 more roundings of 2^-24 of values up to |x1| + |x2|: 2^-20 of that in all."""
    u, tiny = ROUNDOFF[got.dtype], TINY[got.dtype]
    err = (got.detach().cpu().double() - ref).abs()
    bound = u * ref.abs() * (1 + 2.0 ** -10) + 2.0 ** -20 * size + tiny
    worst = (err - bound).max().item() if err.numel() else 0.0
    assert worst <= 0, f"{what}: {worst} above the bound"


def prefix_plain(q, k, v, kp, vp, dout, spans_q, spans_k, n_pre, scale, mask, out_in=None):
    """Forward and backward of shared-prefix attention from the definition, in float64.

    ``spans_*``: (offset, real length) of each sequence. ``out_in``: the forward output the
    backward forms rowsum(dO O) from (default: the exact one). Returns a dict of ``out, lse,
    dq, dk, dv, dkp, dvp`` and, under ``"size"``, for each of them the sums of magnitudes that
    rounding P, dS (and O in D) to 16 bits is relative to, and under ``"flat"`` those that their
    subnormal rounding is."""
    q, k, v, kp, vp, dout = (x.detach().cpu().double() for x in (q, k, v, kp, vp, dout))
    o_in = None if out_in is None else out_in.detach().cpu().double()
    hq, hkv = q.shape[1], k.shape[1]
    G = hq // hkv
    names = {"out": q, "dq": q, "dk": k, "dv": k, "dkp": kp, "dvp": kp}
    R = {n: torch.zeros_like(x) for n, x in names.items()}
    size = {n: torch.zeros_like(x) for n, x in names.items()}
    flat = {n: torch.zeros_like(x) for n, x in names.items()}
    lse = torch.zeros(q.shape[:2], dtype=torch.float64)
    for (oq, n), (ok, m) in zip(spans_q, spans_k):
        if n == 0:
            continue
        see = torch.ones(n, n_pre + m, dtype=torch.bool)
        if mask != "padding":
            diag = m - n if mask == "padding_causal_bottom_right" else 0
            see[:, n_pre:] = torch.arange(m)[None, :] <= torch.arange(n)[:, None] + diag
        for h in range(hq):
            g = h // G
            Q, K = q[oq:oq + n, h], torch.cat((kp[:n_pre, g], k[ok:ok + m, g]))
            V, dO = torch.cat((vp[:n_pre, g], v[ok:ok + m, g])), dout[oq:oq + n, h]
            S = torch.where(see, scale * Q @ K.T, torch.tensor(-math.inf, dtype=torch.float64))
            top = S.max(dim=1, keepdim=True).values if S.shape[1] else torch.full((n, 1), -math.inf, dtype=torch.float64)
            e = torch.where(see, torch.exp(S - torch.where(top == -math.inf, 0.0, top)), 0.0)
            tot = e.sum(1, keepdim=True)
            P = e / torch.where(tot > 0, tot, 1.0)
            O = P @ V
            R["out"][oq:oq + n, h] = O
            lse[oq:oq + n, h] = (top + torch.log(tot))[:, 0]
            size["out"][oq:oq + n, h] = P @ V.abs()
            flat["out"][oq:oq + n, h] = see.double() @ V.abs() / torch.where(tot > 0, tot, 1.0)
            Oi = O if o_in is None else o_in[oq:oq + n, h]
            D = (dO * Oi).sum(1, keepdim=True)
            a = (dO * Oi).abs().sum(1, keepdim=True)  # what a rounded O moves D by, relative
            dS = P * (dO @ V.T - D)
            sd = dS.abs() + (P * a if o_in is None else 0.0)
            f = see.double()
            R["dq"][oq:oq + n, h] = scale * dS @ K
            size["dq"][oq:oq + n, h] = abs(scale) * sd @ K.abs()
            flat["dq"][oq:oq + n, h] = abs(scale) * f @ K.abs()
            for name, pre, x, sx, rows in (("dk", "dkp", scale * dS.T @ Q, abs(scale) * sd.T @ Q.abs(), abs(scale) * f.T @ Q.abs()),
                                           ("dv", "dvp", P.T @ dO, P.T @ dO.abs(), f.T @ dO.abs())):
                R[pre][:n_pre, g] += x[:n_pre]
                R[name][ok:ok + m, g] += x[n_pre:]
                size[pre][:n_pre, g] += sx[:n_pre]
                size[name][ok:ok + m, g] += sx[n_pre:]
                flat[pre][:n_pre, g] += rows[:n_pre]
                flat[name][ok:ok + m, g] += rows[n_pre:]
    return {**R, "lse": lse, "size": size, "flat": flat}


# |x - ref| <= 2 u (size + |ref|) + tiny (flat + 1): the operands P and dS are rounded once
# (u of each term), the result once (u of it), so u (size + |ref|) bounds those in the worst
# case; the other half covers the fp32 accumulation, ex2's 2^-22 and the lse's rounding
# (2^-24 |lse| as a factor on P), all far below u. The largest error over a whole tensor is
# held to the same by norm with 1 u, since independent roundings add in quadrature.
def prefix_check(got, ref, names, dtype, lse_tol=None):
    u, tiny = ROUNDOFF[dtype], TINY[dtype]
    for name in names:
        x = got[name].detach().cpu().double()
        r = ref[name]
        if name == "lse":
            inf = torch.isinf(r)
            assert torch.equal(inf, torch.isinf(x)), "lse: other rows are empty"
            # fp32: 2^-22 of P (ex2) and of |lse|, scores of d products of 2^-24 each
            err = torch.where(inf, 0.0, x - r).abs().max().item()
            assert err <= (1e-4 if lse_tol is None else lse_tol), f"lse off by {err}"
            continue
        err = (x - r).abs()
        bound = 2 * u * (ref["size"][name] + r.abs()) + 4 * tiny * (ref["flat"][name] + 1)
        bound = torch.where(ref["size"][name] + r.abs() > 0, bound, 0.0)  # rows that must be zero are
        over = (err - bound).max().item() if err.numel() else 0.0
        assert not torch.isnan(x).any(), f"{name}: NaN"
        assert over <= 0, f"{name}: {over} above the bound (error {err.max().item()})"
