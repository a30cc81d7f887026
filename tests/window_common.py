"""Plain 64-bit form of sliding-window attention with sinks, for its tests."""

from __future__ import annotations

import math

import torch


def visible(n, m, mask, window, sinks):
    """[n, m] table: query i sees key j."""
    p = torch.arange(n)[:, None] + (m - n if mask == "padding_causal_bottom_right" else 0)
    j = torch.arange(m)[None, :]
    see = j <= p
    return see & ((p - j < window) | (j < sinks)) if window else see


def window_plain(q, k, v, dout, spans_q, spans_k, scale, mask, window, sinks, out_in=None):
    """Forward and backward from the definition, in float64. ``spans_*``: (offset, real length)
    of each sequence. Returns a dict of ``out, lse, dq, dk, dv`` and, under ``"size"``, the sums
    of magnitudes that rounding P, dS (and O in D) to 16 bits is relative to, and under
    ``"flat"`` those that their subnormal rounding is."""
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    back = dout is not None
    dout = dout.detach().cpu().double() if back else None
    o_in = None if out_in is None else out_in.detach().cpu().double()
    hq, hkv = q.shape[1], k.shape[1]
    names = {"out": q, "dq": q, "dk": k, "dv": k} if back else {"out": q}
    R, size, flat = ({n: torch.zeros_like(x) for n, x in names.items()} for _ in range(3))
    lse = torch.zeros(q.shape[:2], dtype=torch.float64)
    for (oq, n), (ok, m) in zip(spans_q, spans_k):
        if n == 0:
            continue
        see = visible(n, m, mask, window, sinks)
        f = see.double()
        for h in range(hq):
            g = h // (hq // hkv)
            Q, K, V = q[oq:oq + n, h], k[ok:ok + m, g], v[ok:ok + m, g]
            S = torch.where(see, scale * Q @ K.T, -math.inf)
            top = S.max(dim=1, keepdim=True).values if m else torch.full((n, 1), -math.inf, dtype=torch.float64)
            e = torch.where(see, torch.exp(S - torch.where(top == -math.inf, 0.0, top)), 0.0)
            tot = e.sum(1, keepdim=True)
            P = e / torch.where(tot > 0, tot, 1.0)
            O = P @ V
            R["out"][oq:oq + n, h] = O
            lse[oq:oq + n, h] = (top + torch.log(tot))[:, 0]
            size["out"][oq:oq + n, h] = P @ V.abs()
            flat["out"][oq:oq + n, h] = f @ V.abs() / torch.where(tot > 0, tot, 1.0)
            if not back:
                continue
            dO = dout[oq:oq + n, h]
            Oi = O if o_in is None else o_in[oq:oq + n, h]
            D = (dO * Oi).sum(1, keepdim=True)
            a = (dO * Oi).abs().sum(1, keepdim=True)  # what a rounded O moves D by, relative
            dS = P * (dO @ V.T - D)
            sd = dS.abs() + (P * a if o_in is None else 0.0)
            R["dq"][oq:oq + n, h] = scale * dS @ K
            size["dq"][oq:oq + n, h] = abs(scale) * sd @ K.abs()
            flat["dq"][oq:oq + n, h] = abs(scale) * f @ K.abs()
            for name, x, sx, rows in (("dk", scale * dS.T @ Q, abs(scale) * sd.T @ Q.abs(), abs(scale) * f.T @ Q.abs()),
                                      ("dv", P.T @ dO, P.T @ dO.abs(), f.T @ dO.abs())):
                R[name][ok:ok + m, g] += x
                size[name][ok:ok + m, g] += sx
                flat[name][ok:ok + m, g] += rows
    return {**R, "lse": lse, "size": size, "flat": flat}
