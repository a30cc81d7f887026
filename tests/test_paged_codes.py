"""The 4-bit cache's steps and codes against exact rational arithmetic, for groups whose differences
32 bits do not hold: a tiny least element, tiny elements far from it, ranges past the largest number."""

from fractions import Fraction

import pytest
import torch

import bwd_packed_varlen_gb300 as ta
from paged_common import four_bits

gpu = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
FORM = {BF: (8, -133), FP: (11, -24)}  # bits of the fraction, exponent of the least number


def _grid(x, dtype):
    """Distance of the type's numbers around x > 0."""
    bits, low = FORM[dtype]
    e = x.numerator.bit_length() - x.denominator.bit_length()  # 2^(e-1) < x < 2^(e+1)
    if Fraction(2) ** e > x:
        e -= 1
    return Fraction(2) ** max(e - bits + 1, low)


def _down(x, dtype):
    return x if x == 0 else x // _grid(x, dtype) * _grid(x, dtype)


def _nearest(x, dtype):
    return x if x == 0 else (round(abs(x) / _grid(abs(x), dtype)) * _grid(abs(x), dtype)) * (1 if x > 0 else -1)


def rational(group, dtype):
    """(step, codes, values) of 32 numbers, from the definition."""
    g = [Fraction(v) for v in group]
    lo, hi = min(g), max(g)
    s = _down((hi - lo) / 15, dtype)
    c = [min(15, round((v - lo) / s)) if s else 0 for v in g]  # (round() of a fraction: ties to even)
    return float(s), c, [float(_nearest(s * k + lo, dtype)) for k in c]


def _rows(dtype, seed):
    """[groups, 32]: kinds of groups that are hard, by turns."""
    gen = torch.Generator().manual_seed(seed)
    up = lambda n: torch.rand(n, 32, generator=gen)  # noqa: E731
    rows = []
    x = up(60) * 16                                          # one-sided, a tiny least element
    x[:, 3] = 1e-6 * (0.2 + up(60)[:, 0])
    rows.append(x)
    x = torch.nn.functional.softplus(8 * torch.randn(60, 32, generator=gen) - 8)
    rows.append(x)
    steps = (torch.arange(32) % 16 * 0.5).repeat(40, 1)      # every border between two codes, and every code
    x = steps + 0.0
    x[:20, 0] = 1e-7 * (1 + up(20)[:, 0])                    # least 1e-7, greatest 7.5: (7.5 - least) / 15 is below 0.5
    x[20:, 0] = -1e-7 * (1 + up(20)[:, 0])
    rows.append(x)
    x = torch.zeros(40, 32)                                  # greatest - least 15 steps of 1, and tiny elements on a border
    x[:, 0], x[:, 1] = -4.5, 10.5
    x[:, 2:] = 1e-6 * torch.randn(40, 30, generator=gen)
    rows.append(x)
    x = torch.randint(0, 31, (40, 32), generator=gen) * 0.5  # borders that are met
    x[:, 0], x[:, 1] = 0, 15
    rows.append(x - torch.randint(-8, 8, (40, 1), generator=gen))
    tiny = float(Fraction(2) ** FORM[dtype][1])
    rows.append(torch.randint(0, 90, (20, 32), generator=gen).double().mul(tiny).float())  # steps of the least numbers
    big = torch.finfo(dtype).max
    x = torch.randn(20, 32, generator=gen).clamp(-1, 1) * big / 2
    x[:, 0], x[:, 1] = big, -big
    x[:10, 2:6] = torch.tensor([0.5, -0.5, 0.1, -0.1])       # nothing beside the range
    rows.append(x)
    return torch.cat(rows).to(dtype)


# ------------------------------------------------------------------ on the CPU
def test_definition_by_hand():
    assert rational([15.0, 1e-7] + [3.0] * 30, BF)[0] == 0.99609375  # (15 - 1e-7) / 15 lies below 1
    assert rational([15.0, -1e-7] + [3.0] * 30, BF)[0] == 1.0
    s, c, v = rational([0.0, 15.0, 0.5, 1.5, 2.5, 2.5000002] + [1.0] * 26, FP)
    assert s == 1.0 and c[:6] == [0, 15, 0, 2, 2, 3] and v[:6] == [0, 15, 0, 2, 2, 3]


@pytest.mark.parametrize("dtype", [BF, FP])
def test_plain_form_where_64_bits_hold_the_differences(dtype):
    x = _rows(dtype, 71)
    x = x[(x.double().abs().amax(1) < 100)]
    codes, meta, _ = four_bits(x)  # (its values are rounded to 32 bits first, which may make a tie)
    for i, g in enumerate(x.double().tolist()):
        s, c, _ = rational(g, dtype)
        assert meta[i, 0, 0].item() == s
        assert [int(b) for b in codes[i]] == [a | b << 4 for a, b in zip(c[0::2], c[1::2])]


# ------------------------------------------------------------------ on the GPU
@gpu
@pytest.mark.parametrize("dtype", [BF, FP])
def test_steps_codes_and_values(dtype):
    x = _rows(dtype, 72)
    n = len(x)
    v = x[:, None].cuda()
    k = -v.flip(0)
    caches = ta.paged_cache((n + 15) // 16, 16, 1, 32, dtype, 4)
    table = torch.arange((n + 15) // 16, dtype=torch.int32, device="cuda")[None]
    cu, past = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ta.paged_append(None, k, v, *caches, table, past, cu, cu)
    held = ta.paged_gather(*caches, table, past, cu, cu, n)
    for new, (codes, meta), got in ((k, *caches[:1], held[0]), (v, *caches[1:], held[1])):
        codes, meta, got = codes.flatten(0, 2)[:n].cpu(), meta.flatten(0, 2)[:n, 0].cpu(), got[:, 0].double().cpu()
        for i, g in enumerate(new[:, 0].double().tolist()):
            s, c, values = rational(g, dtype)
            assert meta[i].tolist() == [s, min(g)], (i, g)
            assert codes[i].tolist() == [a | b << 4 for a, b in zip(c[0::2], c[1::2])], (i, g)
            assert got[i].tolist() == values, (i, g)
