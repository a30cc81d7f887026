"""Plain 64-bit forms of the paged cache's operations, for their tests."""

from __future__ import annotations

import ctypes

import torch


class CacheStruct(ctypes.Structure):
    """te_attn_paged_cache of include/te_attn.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_meta", "v_meta")] +
                [(n, ctypes.c_int64) for n in ("k_stride", "v_stride", "k_meta_stride", "v_meta_stride")] +
                [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64)] +
                [(n, ctypes.c_int) for n in ("num_pages", "page_size", "max_pages", "hkv", "d", "dtype")])


def sound_struct(bits=16, page=16, hkv=2, d=64):
    """A description that passes every check, of memory that is never looked at."""
    row = 2 * d if bits == 16 else d // 2
    c = CacheStruct(k=4096, v=8192, k_stride=row * page * hkv, v_stride=row * page * hkv, page_table=4096, table_stride=4,
                    num_pages=9, page_size=page, max_pages=4, hkv=hkv, d=d, dtype=1)
    if bits == 4:
        c.k_meta, c.v_meta, c.k_meta_stride, c.v_meta_stride = 4096, 4096, d // 8 * page * hkv, d // 8 * page * hkv
    return c


def _down(x, dtype):
    """x >= 0, rounded towards zero to 16 bits, in float64."""
    keep = 8 if dtype == torch.bfloat16 else 11
    m, e = torch.frexp(x)
    ulp = torch.ldexp(torch.ones_like(x), torch.clamp(e - keep, min=-133 if dtype == torch.bfloat16 else -24))
    return torch.floor(x / ulp) * ulp


def four_bits(x):
    """(codes uint8 [..., d / 2], steps and least values [..., d / 32, 2], values [..., d]) of 16-bit
    x [..., d], from the definition in float64. The value is rounded once: s c + m is exact in
    float64 for numbers of like size, and elsewhere the smaller one only decides a tie."""
    g = x.cpu().double().unflatten(-1, (-1, 32))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = _down((hi - lo) / 15, x.dtype)
    c = torch.where(s > 0, torch.round((g - lo) / torch.where(s > 0, s, 1.0)), 0.0).clamp(0, 15)
    value = (s * c + lo).flatten(-2).to(x.dtype)
    c = c.flatten(-2).to(torch.uint8)
    meta = torch.cat((s, lo), dim=-1).to(x.dtype)
    bad = ~torch.isfinite(g).all(-1)
    if bad.any():
        c = torch.where(bad.repeat_interleave(32, -1), torch.zeros_like(c), c)
        meta = torch.where(bad[..., None], torch.full_like(meta, float("nan")), meta)
        value = torch.where(bad.repeat_interleave(32, -1), torch.full_like(value, float("nan")), value)
    return c[..., 0::2] | (c[..., 1::2] << 4), meta, value


def tables(lengths, page, seed, spare=5, width=None):
    """(page table int32 [batch, width], pages in all): each sequence's pages in random order; entries that
    no position needs are out of range."""
    need = [(n + page - 1) // page for n in lengths]
    total = sum(need) + spare
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed))
    width = max(need + [1]) + 1 if width is None else width
    t = torch.full((len(lengths), width), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, total


def places(table, page, past, lengths, offsets):
    """(packed rows, pages, slots) of the new tokens of every sequence."""
    rows, pages, slots = [], [], []
    for b, (p, n, o) in enumerate(zip(past, lengths, offsets)):
        for i in range(n):
            rows.append(o + i)
            pages.append(int(table[b, (p + i) // page]))
            slots.append((p + i) % page)
    return torch.tensor(rows, dtype=torch.long), torch.tensor(pages, dtype=torch.long), torch.tensor(slots, dtype=torch.long)
