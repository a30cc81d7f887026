"""Workloads of sliding-window attention and of the paged key/value cache.

``run`` computes a case either in plain form (elementary torch operations in 32 bits,
rounded once at the end) or, with ``own`` set, through this package's operators.
``exact`` gives the same outputs from the definitions in 64 bits.

Three kinds of case (``op``):

``window``  causal attention of packed sequences in which a query sees the last ``window`` keys
            up to its own position and the first ``sinks`` ones; with ``back`` the gradients too;
``append``  rotation of new queries and keys by their positions, and the new keys and values
            written behind ``past`` tokens of each sequence's pages, in 16 or in 4 bits;
``paged``   attention of new queries over such pages, all keys or a window and sinks.

4 bits: of every 32 neighbouring elements of a head the least, m, and the step s, a 15th of the
range rounded towards zero to 16 bits, are kept, and for each element the whole number c in 0..15
nearest to (x - m) / s; the value that stands for is s c + m, rounded to 16 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GOLDEN = 0.6180339887498949


def listed():
    return [
        # training on short documents: a small step of a narrow model
        {"name": "window_train_small", "op": "window", "back": True, "batch": 5, "q_lo": 20, "q_hi": 300, "past_lo": 0, "past_hi": 0, "window": 48,
         "sinks": 4, "hq": 8, "hkv": 2, "d": 64, "dtype": "fp16", "mask": "padding_causal"},
        # one layer's share of a training step on long packed sequences
        {"name": "window_train", "op": "window", "back": True, "batch": 4, "q_lo": 1500, "q_hi": 6000, "past_lo": 0, "past_hi": 0, "window": 1024,
         "sinks": 4, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16", "mask": "padding_causal"},
        # the next pieces of two long prompts, read in behind what is known
        {"name": "window_prompt", "op": "window", "back": False, "batch": 2, "q_lo": 2000, "q_hi": 4096, "past_lo": 3000, "past_hi": 8000,
         "window": 2000, "sinks": 64, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16", "mask": "padding_causal_bottom_right"},
        # one decoding step of a mid-sized batch
        {"name": "append_step", "op": "append", "bits": 16, "batch": 48, "q_lo": 1, "q_hi": 1, "past_lo": 100, "past_hi": 1500, "page": 16, "hq": 32,
         "hkv": 8, "d": 128, "rot": 128, "interleaved": False, "dtype": "bf16"},
        # prompts that have just been projected
        {"name": "append_prompt", "op": "append", "bits": 16, "batch": 5, "q_lo": 1500, "q_hi": 8000, "past_lo": 0, "past_hi": 200, "page": 64, "hq": 32,
         "hkv": 8, "d": 128, "rot": 128, "interleaved": False, "dtype": "bf16"},
        # shorter prompts into a cache of 4 bits, a part of the head rotated, and the values it then holds for them
        {"name": "append_prompt_4", "op": "append", "bits": 4, "batch": 12, "q_lo": 30, "q_hi": 900, "past_lo": 0, "past_hi": 500, "page": 32, "hq": 16,
         "hkv": 8, "d": 64, "rot": 32, "interleaved": True, "dtype": "fp16"},
        # decoding: the smallest call
        {"name": "step_small", "op": "paged", "bits": 16, "batch": 3, "q_lo": 1, "q_hi": 1, "past_lo": 20, "past_hi": 200, "page": 16, "window": 0,
         "sinks": 0, "hq": 8, "hkv": 8, "d": 64, "dtype": "fp16"},
        # decoding: a usual batch
        {"name": "step_usual", "op": "paged", "bits": 16, "batch": 64, "q_lo": 1, "q_hi": 1, "past_lo": 200, "past_hi": 4000, "page": 16, "window": 0,
         "sinks": 0, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16"},
        # decoding far into long texts through a window
        {"name": "step_window", "op": "paged", "bits": 16, "batch": 32, "q_lo": 1, "q_hi": 1, "past_lo": 8000, "past_hi": 30000, "page": 64,
         "window": 4096, "sinks": 4, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16"},
        # pieces of prompts read in behind what is cached
        {"name": "chunk", "op": "paged", "bits": 16, "batch": 4, "q_lo": 100, "q_hi": 512, "past_lo": 2000, "past_hi": 12000, "page": 64, "window": 0,
         "sinks": 0, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16"},
        # a few drafted tokens of each sequence, some sequences idle
        {"name": "draft_4", "op": "paged", "bits": 4, "batch": 20, "q_lo": 0, "q_hi": 4, "past_lo": 100, "past_hi": 2000, "page": 16, "window": 0,
         "sinks": 0, "hq": 24, "hkv": 4, "d": 96, "dtype": "fp16"},
        # decoding: many sequences with long caches
        {"name": "step_large_4", "op": "paged", "bits": 4, "batch": 128, "q_lo": 1, "q_hi": 1, "past_lo": 1000, "past_hi": 16000, "page": 32, "window": 0,
         "sinks": 0, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm."""
    return min(hi, int(lo * (hi / lo) ** rng.random() + rng.random()))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        lq, lk = _lengths(c)
        dense = c["batch"] * c["hq"] * max(lq) * max(lk)
        if c["op"] == "window" and dense < 4e9 and w["flops"] < (5e11 if c["back"] else 2e12):
            return c
        if c["op"] == "append" and w["bytes"] < 6e8 and c["batch"] * max(lk) * c["hkv"] * c["d"] < 3e8:
            return c
        if c["op"] == "paged" and dense < 3e9 and c["batch"] * max(lk) * c["hkv"] * c["d"] < 1.2e9 and w["flops"] < 2e11:
            return c


def _draw(rng):
    hkv = rng.choice((1, 2, 4, 8))
    c = {"op": rng.choice(("window", "append", "paged", "paged")), "dtype": rng.choice(("bf16", "fp16")), "hkv": hkv,
         "hq": hkv * rng.choice((1, 2, 3, 4, 6, 8))}
    if c["op"] == "window":
        hi, past = _log(rng, 20, 6000), rng.choice((0, _log(rng, 10, 8000)))
        c.update(back=rng.random() < 0.6, batch=_log(rng, 1, 24), q_lo=hi // 5, q_hi=hi, past_lo=past // 3, past_hi=past, window=_log(rng, 1, 4096),
                 sinks=rng.choice((0, 1, 4, _log(rng, 5, 300))), d=rng.choice((32, 64, 80, 96, 128, 128, 256)),
                 mask="padding_causal_bottom_right" if past else "padding_causal")
        return c
    c["bits"] = rng.choice((16, 4))
    c["d"] = rng.choice((64, 96, 128, 128, 256) if c["bits"] == 4 else (64, 80, 96, 128, 128, 256))
    c["page"] = rng.choice((16, 32, 64, 128))
    if c["op"] == "append":
        hi, past, d = rng.choice((1, _log(rng, 2, 8000))), _log(rng, 1, 20000), c["d"]
        c.update(batch=_log(rng, 1, 128), q_lo=hi // 5, q_hi=hi, past_lo=past // 4, past_hi=past, rot=rng.choice((d, d // 2, d // 4)) // 2 * 2,
                 interleaved=rng.random() < 0.5)
        return c
    many = rng.random() < 0.4
    hi, past = _log(rng, 2, 600) if many else 1, _log(rng, 10, 30000)
    c.update(batch=_log(rng, 1, 16 if many else 160), q_lo=hi // 6 if many else 1, q_hi=hi, past_lo=past // 5, past_hi=past,
             window=rng.choice((0, 0, _log(rng, 16, 5000))))
    c["sinks"] = rng.choice((0, 4, 20)) if c["window"] else 0
    return c


def _spread(n, lo, hi, step=GOLDEN):
    """n lengths in [lo, hi], the same for every seed, the first of them the longest."""
    return [hi - int(((i * step) % 1.0) * (hi - lo + 1)) for i in range(n)]


def _lengths(case):
    """(new tokens, keys) of each sequence."""
    lq = _spread(case["batch"], case["q_lo"], case["q_hi"])
    past = _spread(case["batch"], case["past_lo"], case["past_hi"], 1 - GOLDEN * GOLDEN * GOLDEN)
    return lq, [a + b for a, b in zip(lq, past)]


def _seen(n, m, diag, window, sinks):
    """(visible pairs, keys that some query sees) of n queries and m keys."""
    pairs = keys = top = 0  # top: keys below it are counted already
    for i in range(n):
        hi = min(m, i + diag + 1)
        if hi <= 0:
            continue
        lo = max(0, i + diag + 1 - window) if window else 0
        first = min(sinks, lo, hi)
        pairs += hi - lo + first if hi > lo else first
        if hi > lo:
            keys += hi - max(lo, top) + (first if top == 0 else 0)
            top = max(top, hi)
    return pairs, keys


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lq, lk = _lengths(case)
    q = 2 * sum(lq) * hq * d
    if case["op"] == "append":
        kv = 2 * 2 * sum(lq) * hkv * d
        cached = kv if case["bits"] == 16 else kv * 5 // 16 * 2 + kv
        return {"bytes": 2 * q + kv + cached, "flops": 3 * sum(lq) * (hq + hkv) * case["rot"]}
    low = case.get("mask") != "padding_causal"
    seen = [_seen(n, m, m - n if low else 0, case["window"], case["sinks"]) for n, m in zip(lq, lk)]
    flops = 4 * d * hq * sum(s[0] for s in seen)
    if case["op"] == "paged":
        kv = 4 * sum(s[1] for s in seen) * hkv * d
        return {"bytes": 2 * q + 4 * sum(lq) * hq + (kv if case["bits"] == 16 else kv * 5 // 16), "flops": flops}
    kv = 4 * sum(lk) * hkv * d
    if case["back"]:
        return {"bytes": 4 * q + 2 * kv + 4 * sum(lq) * hq, "flops": 3.5 * flops}
    return {"bytes": 2 * q + kv + 4 * sum(lq) * hq, "flops": flops}


def _offsets(lengths, slot):
    """Prefix sums of the lengths and of the slots they are kept in."""
    real, padded = [0], [0]
    for n in lengths:
        real.append(real[-1] + n)
        padded.append(padded[-1] + (n + slot - 1) // slot * slot)
    return real, padded


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(gen, shape, dtype, spread=None):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x if spread is None else x * spread).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, hq, hkv, d, batch = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["d"], case["batch"]
    lq, lk = _lengths(case)
    rq, pq = _offsets(lq, 1 if case["q_hi"] == 1 else 8)
    wide = torch.exp(0.4 * torch.randn(d, generator=gen, device="cuda"))  # channels differ in size
    s = {"case": case, "lq": lq, "lk": lk, "cu_q": _ints(rq), "cu_q_pad": _ints(pq), "pq": pq, "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "window":
        rk, pk = _offsets(lk, 8)
        s.update(cu_k=_ints(rk), cu_k_pad=_ints(pk), pk=pk, q=_normal(gen, (pq[-1], hq, d), dtype, wide), k=_normal(gen, (pk[-1], hkv, d), dtype),
                 v=_normal(gen, (pk[-1], hkv, d), dtype))
        if case["back"]:
            s["dout"] = _normal(gen, (pq[-1], hq, d), dtype)
        return s
    # pages in the order in which requests came and went, some of them free; a page's tail holds what was there before
    page = case["page"]
    need = [(n + page - 1) // page for n in lk]
    order = torch.randperm(sum(need) + 7, generator=gen, device="cuda").int()
    width = max(need) + 1
    at, own_pages = [0], torch.zeros(batch, width, dtype=torch.int32, device="cuda")
    for n in need:
        at.append(at[-1] + n)
    column = torch.arange(width, device="cuda")
    starts, counts = _ints(at[:-1])[:, None], _ints(need)[:, None]
    own_pages = torch.where(column < counts, order[(starts + torch.minimum(column, counts - 1).clamp(min=0)).long()], 0).int()
    shape = (sum(need) + 7, hkv, page, d)
    s.update(pages=own_pages.contiguous(), past=_ints([b - a for a, b in zip(lq, lk)]), total=pq[-1])
    if case["op"] == "append":
        # queries, keys and values are slices of one projection's output, as a layer has them
        qkv = _normal(gen, (pq[-1], hq + 2 * hkv, d), dtype)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
        s["freq"] = 10000.0 ** (-2.0 * torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64) / case["rot"])
        caches = [torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2)]
    else:
        s["q"] = _normal(gen, (pq[-1], hq, d), dtype, wide)
        caches = [_normal(gen, shape, dtype) for _ in range(2)]
    s["kc"], s["vc"] = caches if case["bits"] == 16 else [_packed(x) for x in caches]
    return s


def _packed(x):
    """_pack(*_codes(x)) a part at a time: large caches in 64 bits would not fit beside each other."""
    parts = [_pack(*_codes(y)) for y in x.split(max(1, (1 << 27) // x[0].numel()))]
    return tuple(torch.cat(y) for y in zip(*parts))


def run(s):
    case = s["case"]
    if own:
        import bwd_packed_varlen_gb300 as ta
        if case["op"] == "window":
            cu = (s["cu_q"], s["cu_k"], s["cu_q_pad"], s["cu_k_pad"])
            out, lse = ta.window_fwd(s["q"], s["k"], s["v"], *cu, s["scale"], case["window"], case["sinks"], case["mask"])
            if not case["back"]:
                return out, lse
            return (out, lse) + tuple(ta.window_bwd(s["q"], s["k"], s["v"], out, s["dout"], lse, *cu, s["scale"], case["window"], case["sinks"],
                                                    case["mask"]))
        cache = (s["kc"], s["vc"], s["pages"], s["past"], s["cu_q"], s["cu_q_pad"])
        if case["op"] == "paged":
            return ta.paged_fwd(s["q"], *cache, s["scale"], window=case["window"], sinks=case["sinks"])
        q = ta.paged_append(s["q"], s["k"], s["v"], *cache, inv_freq=s["freq"], interleaved=case["interleaved"])
        return (q, s["kc"], s["vc"]) if case["bits"] == 16 else (q,) + tuple(ta.paged_gather(*cache, s["total"]))
    return {"window": _plain_window, "append": _plain_append, "paged": _plain_paged}[case["op"]](s)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _towards_zero(x, dtype):
    """x >= 0 (64 bits), rounded towards zero to 16 bits."""
    y = x.to(dtype)
    return torch.where(y.double() > x, (y.view(torch.int16) - 1).view(dtype), y)


def _codes(x):
    """(codes, steps, least values) of 16-bit x [..., d], in groups of 32; in 64 bits, for what lies next to a border."""
    g = x.double().unflatten(-1, (-1, 32))
    least = g.amin(dim=-1)
    step = _towards_zero((g.amax(dim=-1) - least) / torch.full_like(least, 15.0), x.dtype)
    wide = step.double()[..., None]
    c = torch.where(wide > 0, torch.round((g - least[..., None]) / torch.where(wide > 0, wide, 1.0)), 0.0).clamp(0, 15)
    return c.flatten(-2).to(torch.uint8), step, least.to(x.dtype)


def _values(codes, step, least):
    """What the codes stand for, in 16 bits."""
    g = codes.float().unflatten(-1, (-1, 32))
    return (g * step.float()[..., None] + least.float()[..., None]).flatten(-2).to(step.dtype)


def _pack(codes, step, least):
    """The cache's form: two codes a byte, the earlier one in the low half; step and least value side by side."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4), torch.stack((step, least), dim=-1)


def _unpack(cache):
    codes, pair = cache
    return torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2), pair[..., 0], pair[..., 1]


def _rows(cu, cu_pad, longest):
    """Tensor rows of every sequence's tokens as a [batch, longest] table, and which of its places are real."""
    i = torch.arange(longest, device="cuda")
    real = i[None, :] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(real, cu_pad[:-1, None] + i[None, :], 0).long(), real


def _plain_append(s):
    case, rot, page = s["case"], s["case"]["rot"], s["case"]["page"]
    rows = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    b = (torch.searchsorted(s["cu_q_pad"], rows, right=True) - 1).clamp(0, case["batch"] - 1)
    i = rows - s["cu_q_pad"][b]
    real = i < (s["cu_q"][1:] - s["cu_q"][:-1])[b]
    pos = s["past"][b] + i
    # angles of far positions, and what lies next to a border between codes, need 64 bits
    angle = pos.double()[:, None] * s["freq"][None, :]
    cos, sin = angle.cos()[:, None, :], angle.sin()[:, None, :]

    def turn(x):
        y = x.double()
        if case["interleaved"]:
            a, c = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack((a * cos - c * sin, c * cos + a * sin), dim=-1).flatten(-2)
        else:
            a, c = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat((a * cos - c * sin, c * cos + a * sin), dim=-1)
        z = torch.cat((z, y[..., rot:]), dim=-1)
        return torch.where(real[:, None, None], z, 0.0).to(x.dtype)

    q, k, v = turn(s["q"]), turn(s["k"]), torch.where(real[:, None, None], s["v"], 0)
    where = s["pages"][b[real], (pos[real] // page).long()].long(), slice(None), (pos[real] % page).long()
    if case["bits"] == 16:
        s["kc"][where], s["vc"][where] = k[real], v[real]
        return q, s["kc"], s["vc"]
    ck, cv = _codes(k), _codes(v)
    for cache, c in ((s["kc"], ck), (s["vc"], cv)):
        for held, new in zip(cache, _pack(*c)):
            held[where] = new[real]
    return q, _values(*ck), _values(*cv)


def _whole(x, like, rows, real):
    y = torch.zeros_like(like)
    y[rows[real]] = x[real].to(like.dtype)
    return y


def _attend(s, q, k, v, edge, real_q):
    """Attention of q [batch, hkv, queries x group, d] over k, v [batch, hkv, keys, d]; edge: the last key of each query."""
    case = s["case"]
    group, j = case["hq"] // case["hkv"], torch.arange(k.shape[2], device="cuda")
    see = j <= edge[..., None]
    if case["window"]:
        see = see & ((edge[..., None] - j < case["window"]) | (j < case["sinks"]))
    see = (see & real_q[..., None])[:, None, :, None, :].expand(-1, 1, -1, group, -1).flatten(2, 3)
    score = torch.where(see, q @ k.transpose(-1, -2) * s["scale"], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    del score
    total = p.sum(dim=-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    return p, p @ v, (top + torch.log(total))[..., 0]


def _plain_window(s):
    case = s["case"]
    hq, hkv, d, batch = case["hq"], case["hkv"], case["d"], case["batch"]
    group, nq, nk = hq // hkv, max(s["lq"]), max(s["lk"])
    iq, real_q = _rows(s["cu_q"], s["cu_q_pad"], nq)
    ik, real_k = _rows(s["cu_k"], s["cu_k_pad"], nk)

    def by_head(x):  # [batch, hkv, queries x group, d]
        return x[iq].float().view(batch, nq, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, nq * group, d)

    def tokens(x):  # back to [batch, queries, hq, ...]
        return x.view((batch, hkv, nq, group) + x.shape[3:]).transpose(1, 2).flatten(2, 3)

    q = by_head(s["q"])
    k, v = (torch.where(real_k[:, None, :, None], s[n][ik].float().permute(0, 2, 1, 3), 0.0) for n in ("k", "v"))
    edge = torch.arange(nq, device="cuda")[None, :].expand(batch, nq)
    lens_q, lens_k = ((c[1:] - c[:-1])[:, None] for c in (s["cu_q"], s["cu_k"]))
    if case["mask"] == "padding_causal_bottom_right":
        edge = edge + lens_k - lens_q
    p, o, lse = _attend(s, q, k, v, edge, real_q)
    out = _whole(tokens(o), s["q"], iq, real_q)
    lse = _whole(tokens(lse), torch.zeros(s["q"].shape[:2], device="cuda"), iq, real_q)
    if not case["back"]:
        return out, lse
    g = by_head(s["dout"])
    dv = p.transpose(-1, -2) @ g
    ds = p * (g @ v.transpose(-1, -2) - (g * o).sum(dim=-1, keepdim=True)) * s["scale"]
    del p
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    dk, dv = (_whole(x.transpose(1, 2), s["k"], ik, real_k) for x in (dk, dv))
    return out, lse, _whole(tokens(dq), s["q"], iq, real_q), dk, dv


def _plain_paged(s):
    case, page = s["case"], s["case"]["page"]
    hq, hkv, d, batch = case["hq"], case["hkv"], case["d"], case["batch"]
    group, nq, nk = hq // hkv, max(s["lq"]), max(s["lk"])
    iq, real_q = _rows(s["cu_q"], s["cu_q_pad"], nq)
    lens_q = s["cu_q"][1:] - s["cu_q"][:-1]
    j = torch.arange(nk, device="cuda")
    real_k = j[None, :] < (s["past"] + lens_q)[:, None]
    where = torch.where(real_k, s["pages"][:, j // page], 0).long()[:, None, :], torch.arange(hkv, device="cuda")[None, :, None], (j % page)[None, None, :]

    def cached(c):  # [batch, hkv, keys, d]
        x = c[where] if case["bits"] == 16 else _values(*_unpack([part[where] for part in c]))
        return torch.where(real_k[:, None, :, None], x.float(), 0.0)

    q = s["q"][iq].float().view(batch, nq, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, nq * group, d)
    edge = s["past"][:, None] + torch.arange(nq, device="cuda")[None, :]
    _, o, lse = _attend(s, q, cached(s["kc"]), cached(s["vc"]), edge, real_q)

    def tokens(x):
        return x.view((batch, hkv, nq, group) + x.shape[3:]).transpose(1, 2).flatten(2, 3)

    return _whole(tokens(o), s["q"], iq, real_q), _whole(tokens(lse), torch.zeros(s["q"].shape[:2], device="cuda"), iq, real_q)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _exact_values(x):
    """What a 4-bit cache gives back for 16-bit x, by going through the sixteen values of each group."""
    g = x.double().unflatten(-1, (-1, 32))
    low, high = g.min(dim=-1, keepdim=True).values, g.max(dim=-1, keepdim=True).values
    fifteenth = (high - low) / torch.full_like(low, 15.0)  # (a true division)
    drop = 53 - (8 if x.dtype == torch.bfloat16 else 11)  # bits of the fraction that the step does not keep
    step = ((fifteenth.view(torch.int64) >> drop) << drop).view(torch.float64)
    if x.dtype == torch.float16:  # below 2^-14 its numbers are multiples of 2^-24
        step = torch.where(fifteenth < 2.0 ** -14, torch.floor(fifteenth * 2.0 ** 24) * 2.0 ** -24, step)
    c = torch.where(step > 0, torch.round((g - low) / torch.where(step > 0, step, torch.ones_like(step))), torch.zeros_like(g))
    return (low + step * c.clamp(max=15)).flatten(-2).to(x.dtype).double()


def _exact_append(s):
    case, rot, page = s["case"], s["case"]["rot"], s["case"]["page"]
    past, table = s["past"].tolist(), s["pages"].long()
    turned = {}
    for name in ("q", "k", "v"):
        x = s[name]
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lq"]):
            rows = slice(s["pq"][b], s["pq"][b] + n)
            z = x[rows].double()
            y[rows] = z
            if name == "v" or n == 0:
                continue
            pair = z[..., :rot].unflatten(-1, (-1, 2)) if case["interleaved"] else z[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
            pos = torch.arange(past[b], past[b] + n, device="cuda", dtype=torch.float64)
            angle = (pos[:, None] * s["freq"])[:, None, :]
            w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(angle), angle))
            y[rows, :, :rot] = w.flatten(-2) if case["interleaved"] else w.transpose(-1, -2).flatten(-2)
        turned[name] = y
    if case["bits"] == 4:
        return (turned["q"],) + tuple(_exact_values(turned[n].to(DTYPES[case["dtype"]])) for n in ("k", "v"))
    caches = []
    for cache, y in ((s["kc"], turned["k"]), (s["vc"], turned["v"])):
        c = cache.double()
        for b, n in enumerate(s["lq"]):
            for i in range(0, n, 4096):
                at = torch.arange(past[b] + i, past[b] + min(n, i + 4096), device="cuda")
                c[table[b, at // page], :, at % page] = y[s["pq"][b] + i:s["pq"][b] + min(n, i + 4096)]
        caches.append(c)
    return (turned["q"], *caches)


def _exact_attention(s):
    case = s["case"]
    hq, hkv, d, window, sinks = case["hq"], case["hkv"], case["d"], case["window"], case["sinks"]
    back = case.get("back", False)
    names = ("q", "k", "v") if back else ("q",)
    grads = {n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in names}
    out, lse = torch.zeros_like(grads["q"]), torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(s["lq"], s["lk"])):
        if n == 0:
            continue
        rq = slice(s["pq"][b], s["pq"][b] + n)
        if case["op"] == "window":
            rk = slice(s["pk"][b], s["pk"][b] + m)
            k, v = s["k"][rk].double(), s["v"][rk].double()
        else:
            k, v = (_cached(c, s["pages"][b], m, case) for c in (s["kc"], s["vc"]))
        leaves = [s["q"][rq].double(), k, v]
        if back:
            leaves = [x.detach().requires_grad_() for x in leaves]
        q4 = leaves[0].view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
        shift = 0 if case.get("mask") == "padding_causal" else m - n
        blocked = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(1 + shift)
        if window:
            early = torch.ones(n, m, dtype=torch.bool, device="cuda").tril(shift - window)
            early[:, :sinks] = False
            blocked |= early
        score = (torch.matmul(q4, leaves[1].permute(1, 2, 0)) * s["scale"]).view(hkv, hq // hkv, n, m).masked_fill(blocked, -math.inf)
        o = torch.matmul(torch.softmax(score, dim=-1).view(hkv, -1, m), leaves[2].transpose(0, 1)).view(hq, n, d).transpose(0, 1)
        out[rq] = o.detach()
        lse[rq] = torch.logsumexp(score.detach(), dim=-1).reshape(hq, n).t()
        if back:
            for name, rows, x in zip(names, (rq, rk, rk), torch.autograd.grad(o, leaves, s["dout"][rq].double())):
                grads[name][rows] = x
    return (out, lse) + (tuple(grads[n] for n in names) if back else ())


def _cached(cache, pages, m, case):
    """Keys or values of one sequence, [m, hkv, d] in 64 bits."""
    ids = pages[:(m + case["page"] - 1) // case["page"]].long()

    def flat(x):
        return x[ids].transpose(1, 2).flatten(0, 1)[:m]

    if case["bits"] == 16:
        return flat(cache).double()
    codes, pair = (flat(x) for x in cache)
    c = torch.stack((codes % 16, codes // 16), dim=-1).flatten(-2).double().unflatten(-1, (-1, 32))
    return (c * pair[..., :1].double() + pair[..., 1:].double()).flatten(-2).to(pair.dtype).double()
