"""Shared-prefix attention by the norm of its errors, which a term that is lost or counted
twice shows in where the bound on single elements is too wide for it."""

import math

import pytest
import torch

from prefix_common import ROUNDOFF, TINY
from test_prefix import ALL, BR, PAD, TL, Case

gpu = pytest.mark.gpu


def _reference(c, out):
    """Results in float64 from the definition, with rowsum(dO O) of the output that the backward
    is given, and for each of their elements the sum of squares of the terms whose operand (P or
    dS) is rounded to 16 bits, and of those terms' other factors."""
    q, k, v, kp, vp, dout, o_in = (x.double() for x in (*c.on, c.dout_on, out))
    hq, hkv, G = q.shape[1], k.shape[1], q.shape[1] // k.shape[1]
    like = {"out": q, "dq": q, "dk": k, "dv": k, "dkp": kp, "dvp": kp}
    ref, terms, flat = ({n: torch.zeros_like(x) for n, x in like.items()} for _ in range(3))
    n_pre = c.prefix
    for (oq, n), (ok, m) in zip(c.spans_q, c.spans_k):
        if n == 0:
            continue
        see = torch.ones(n, n_pre + m, dtype=torch.bool, device="cuda")
        if c.mask != PAD:
            see[:, n_pre:] = torch.ones(n, m, dtype=torch.bool, device="cuda").tril(m - n if c.mask == BR else 0)
        for h in range(hq):
            g = h // G
            K, V = torch.cat((kp[:n_pre, g], k[ok:ok + m, g])), torch.cat((vp[:n_pre, g], v[ok:ok + m, g]))
            Q, dO = q[oq:oq + n, h], dout[oq:oq + n, h]
            P = torch.softmax((c.scale * Q @ K.T).masked_fill(~see, -math.inf), dim=1)
            dS = P * (dO @ V.T - (dO * o_in[oq:oq + n, h]).sum(1, keepdim=True))
            f = see.double()
            for name, left, right in (("out", P, V), ("dq", c.scale * dS, K)):
                ref[name][oq:oq + n, h] = left @ right
                terms[name][oq:oq + n, h] = left ** 2 @ right ** 2
                flat[name][oq:oq + n, h] = f @ right ** 2
            for own, pre, left, right in (("dk", "dkp", c.scale * dS, Q), ("dv", "dvp", P, dO)):
                for x, a, b in ((ref, left, right), (terms, left ** 2, right ** 2), (flat, f, right ** 2)):
                    y = a.T @ b
                    x[pre][:n_pre, g] += y[:n_pre]
                    x[own][ok:ok + m, g] += y[n_pre:]
    return ref, terms, flat


@gpu
@pytest.mark.parametrize("d,hq,hkv,dtype,mask,prefix,lq,extra", [
    (128, 8, 2, torch.bfloat16, TL, 300, [500, 1, 233, 700, 64], 0),      # the prefix's sweep in parts
    (64, 6, 1, torch.float16, BR, 150, [90, 40, 0, 77, 128, 5, 33], 60),
    (256, 4, 2, torch.bfloat16, PAD, 260, [130, 300, 9], 40),
    (80, 12, 4, torch.bfloat16, TL, 615, [38, 192, 100, 61] * 4, 0),
    (96, 8, 1, torch.float16, BR, 40, [200, 3, 150], 900),
    (128, 4, 4, torch.bfloat16, TL, 9000, [300, 200], 0)])                # and whole, over many key tiles
def test_errors_in_the_mean(d, hq, hkv, dtype, mask, prefix, lq, extra):
    """P and dS are rounded once each to 16 bits, to within u of a term and as likely up as down,
    and the result once, to within u of it. Such errors add in quadrature: their norm is at most
    u times that of the terms and results, taken as if every one were the largest possible (on
    average one is 0.4 of that, which leaves fp32's own, below 2^-20, ample room). Values below
    the type's normal range are off by up to `tiny` instead."""
    c = Case(d + prefix, lq, [n + (extra * (i + 1)) // len(lq) for i, n in enumerate(lq)], prefix, hq, hkv, d, dtype, mask).dev()
    out, lse = c.fwd()
    got = {"out": out, **dict(zip(ALL, c.bwd(out, lse)))}
    ref, terms, flat = _reference(c, out)
    u, tiny = ROUNDOFF[dtype], TINY[dtype]
    for name, x in got.items():
        err = (x.double() - ref[name]).norm().item()
        bound = math.sqrt((u * u * (terms[name] + ref[name] ** 2) + tiny * tiny * (flat[name] + 1)).sum().item())
        assert err <= bound, f"{name}: {err} above {bound}"
