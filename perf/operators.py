"""Workloads of the rotary-position and shared-prefix attention operators.

``run`` computes a case either in plain form (elementary torch operations in 32 bits,
rounded once at the end) or, with ``own`` set, through this package's operators.
``exact`` gives the same outputs from the definitions in 64 bits.

Three kinds of case (``op``):

``rope``    rotation of the queries and keys of packed sequences by their positions,
            or of their gradients by the negative angle (``back``);
``attend``  attention of packed queries over keys that every sequence shares (the
            prefix) followed by the sequence's own; ``q_hi`` 1 is a decoding step;
``train``   such an attention forward and backward, the prefix's gradients summed
            over the sequences.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GOLDEN = 0.6180339887498949


def listed():
    return [
        # one decoding step of a mid-sized batch: a token per sequence, far positions
        {"name": "rope_step", "op": "rope", "back": False, "batch": 48, "lo": 1, "hi": 1, "slot": 1, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "dtype": "bf16", "start": 130000, "scaled": True},
        # a training batch of long packed sequences
        {"name": "rope_train", "op": "rope", "back": False, "batch": 7, "lo": 700, "hi": 8100, "slot": 64, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "dtype": "bf16", "start": 0, "scaled": True},
        # its counterpart on the way back, with a part of the head rotated in neighbouring pairs
        {"name": "rope_back_part", "op": "rope", "back": True, "batch": 33, "lo": 0, "hi": 500, "slot": 8, "hq": 32, "hkv": 32, "d": 80,
         "rot": 32, "interleaved": True, "dtype": "fp16", "start": 2000, "scaled": False},
        # decoding: the smallest call
        {"name": "step_small", "op": "attend", "batch": 3, "q_lo": 1, "q_hi": 1, "past_lo": 0, "past_hi": 40, "prefix": 200, "hq": 8,
         "hkv": 8, "d": 64, "dtype": "fp16", "mask": "padding_causal_bottom_right"},
        # decoding: a usual batch behind a long instruction
        {"name": "step_usual", "op": "attend", "batch": 48, "q_lo": 1, "q_hi": 1, "past_lo": 30, "past_hi": 1000, "prefix": 6000, "hq": 32,
         "hkv": 8, "d": 128, "dtype": "bf16", "mask": "padding_causal_bottom_right"},
        # decoding: many sequences behind a long document
        {"name": "step_large", "op": "attend", "batch": 256, "q_lo": 1, "q_hi": 1, "past_lo": 256, "past_hi": 4000, "prefix": 32768, "hq": 32,
         "hkv": 8, "d": 128, "dtype": "bf16", "mask": "padding_causal_bottom_right"},
        # decoding: wide heads
        {"name": "step_wide", "op": "attend", "batch": 24, "q_lo": 1, "q_hi": 1, "past_lo": 100, "past_hi": 900, "prefix": 20000, "hq": 16,
         "hkv": 2, "d": 256, "dtype": "bf16", "mask": "padding_causal_bottom_right"},
        # a few drafted tokens for each sequence, some sequences idle
        {"name": "draft", "op": "attend", "batch": 20, "q_lo": 0, "q_hi": 7, "past_lo": 50, "past_hi": 700, "prefix": 2500, "hq": 24,
         "hkv": 4, "d": 96, "dtype": "fp16", "mask": "padding_causal_bottom_right"},
        # questions of many users about one document, read in
        {"name": "read_in", "op": "attend", "batch": 12, "q_lo": 150, "q_hi": 1400, "past_lo": 0, "past_hi": 300, "prefix": 5000, "hq": 32,
         "hkv": 8, "d": 128, "dtype": "bf16", "mask": "padding_causal_bottom_right"},
        # training on several continuations of one prompt: small
        {"name": "train_small", "op": "train", "batch": 5, "q_lo": 20, "q_hi": 110, "past_lo": 0, "past_hi": 0, "prefix": 150, "hq": 8,
         "hkv": 2, "d": 64, "dtype": "fp16", "mask": "padding_causal"},
        # and a full step's share of one layer
        {"name": "train_large", "op": "train", "batch": 16, "q_lo": 200, "q_hi": 900, "past_lo": 0, "past_hi": 0, "prefix": 3500, "hq": 32,
         "hkv": 8, "d": 128, "dtype": "bf16", "mask": "padding_causal"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm."""
    return min(hi, int(lo * (hi / lo) ** rng.random() + rng.random()))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if c["op"] == "rope" and w["bytes"] < 1.3e9:
            return c
        if c["op"] == "attend" and w["bytes"] < 2.5e9 and w["flops"] < 1.2e12:
            return c
        if c["op"] == "train" and w["flops"] < 2.2e12:
            return c


def _draw(rng):
    hkv = rng.choice((1, 2, 4, 8))
    c = {"op": rng.choice(("rope", "attend", "attend", "train")), "dtype": rng.choice(("bf16", "fp16")), "hkv": hkv}
    if c["op"] == "rope":
        group, d = rng.choice((1, 2, 3, 4, 6, 8)), rng.choice((32, 48, 64, 80, 96, 128, 256))
        hi = _log(rng, 1, 8000)
        c.update(back=rng.random() < 0.4, batch=_log(rng, 1, 64), lo=rng.choice((0, hi // 3, hi)), hi=hi, slot=rng.choice((1, 8, 64)),
                 hq=hkv * group, d=d, rot=rng.choice((d, d // 2, d // 4)) // 2 * 2, interleaved=rng.random() < 0.5,
                 start=rng.choice((0, _log(rng, 100, 1000000))), scaled=rng.random() < 0.5)
        c["lo"] = max(1, c["lo"]) if c["batch"] == 1 else c["lo"]
        return c
    c.update(hq=hkv * rng.choice((1, 2, 4, 6, 8)), d=rng.choice((64, 64, 80, 96, 128, 128, 128, 256)))
    if c["op"] == "attend":
        many = rng.random() < 0.35
        hi = _log(rng, 2, 1400) if many else 1
        past = _log(rng, 8, 4000)
        c.update(batch=_log(rng, 1, 32 if many else 256), q_lo=hi // 8 if many else 1, q_hi=hi, past_lo=past // 6, past_hi=past,
                 prefix=_log(rng, 100, 8000 if many else 40000), mask=rng.choice(("padding_causal_bottom_right",) * 3 + ("padding",)))
    else:
        hi = _log(rng, 30, 1000)
        c.update(batch=_log(rng, 2, 24), q_lo=hi // 5, q_hi=hi, past_lo=0, past_hi=0, prefix=_log(rng, 100, 4500), mask="padding_causal")
    return c


def _spread(n, lo, hi, step=GOLDEN):
    """n lengths in [lo, hi], the same for every seed, the first of them the longest."""
    return [hi - int(((i * step) % 1.0) * (hi - lo + 1)) for i in range(n)]


def _lengths(case):
    """(query lengths, own key lengths) of an attention case."""
    lq = _spread(case["batch"], case["q_lo"], case["q_hi"])
    past = _spread(case["batch"], case["past_lo"], case["past_hi"], 1 - GOLDEN * GOLDEN * GOLDEN)
    return lq, [a + b for a, b in zip(lq, past)]


def _visible(case):
    """Own (query, key) pairs that the mask leaves, over all sequences."""
    lq, lk = _lengths(case)
    if case["mask"] == "padding":
        return sum(a * b for a, b in zip(lq, lk))
    if case["mask"] == "padding_causal":
        return sum(sum(min(i + 1, b) for i in range(a)) for a, b in zip(lq, lk))
    return sum(sum(max(0, b - a + i + 1) for i in range(a)) for a, b in zip(lq, lk))


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        tokens = sum(_spread(case["batch"], case["lo"], case["hi"]))
        return {"bytes": 4 * tokens * (hq + hkv) * d, "flops": 3 * tokens * (hq + hkv) * case["rot"]}
    lq, lk = _lengths(case)
    q, kv = 2 * sum(lq) * hq * d, 4 * (sum(lk) + case["prefix"]) * hkv * d
    flops = 4 * d * hq * (sum(lq) * case["prefix"] + _visible(case))
    if case["op"] == "attend":
        return {"bytes": 2 * q + kv + 4 * sum(lq) * hq, "flops": flops}
    return {"bytes": 4 * q + 2 * kv + 4 * sum(lq) * hq, "flops": 3.5 * flops}


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


def _frequencies(case):
    """Angle per position of each rotated pair (64 bits) and the factor on the result; scaled: long wavelengths are
    stretched eightfold, short ones kept, with a ramp between them."""
    n = case["rot"] // 2
    w = [10000.0 ** (-2.0 * i / case["rot"]) for i in range(n)]
    if not case["scaled"]:
        return w, 1.0
    out = []
    for x in w:
        turns = 4096 * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31.0))
        out.append(x * keep + x / 8.0 * (1 - keep))
    return out, 0.1 * math.log(8.0) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, hq, hkv, d, batch = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["d"], case["batch"]
    if case["op"] == "rope":
        lengths = _spread(batch, case["lo"], case["hi"])
        real, padded = _offsets(lengths, case["slot"])
        # queries and keys are slices of one projection's output, as a layer has them
        qkv = _normal(gen, (padded[-1], hq + 2 * hkv, d), dtype)
        freq, mscale = _frequencies(case)
        start = _spread(batch, case["start"] // 2, case["start"])
        return {"case": case, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "cu": _ints(real), "cu_pad": _ints(padded), "start": _ints(start),
                "freq": torch.tensor(freq, dtype=torch.float64, device="cuda"), "mscale": mscale, "lengths": lengths}
    lq, lk = _lengths(case)
    rq, pq = _offsets(lq, 1 if case["q_hi"] == 1 else 8)
    rk, pk = _offsets(lk, 64 if case["op"] == "attend" else 8)
    wide = torch.exp(0.4 * torch.randn(d, generator=gen, device="cuda"))  # channels differ in size
    s = {"case": case, "lq": lq, "lk": lk, "scale": 1.0 / math.sqrt(d), "cu_q": _ints(rq), "cu_k": _ints(rk), "cu_q_pad": _ints(pq),
         "cu_k_pad": _ints(pk), "pq": pq, "pk": pk,
         "q": _normal(gen, (pq[-1], hq, d), dtype, wide), "k": _normal(gen, (pk[-1], hkv, d), dtype), "v": _normal(gen, (pk[-1], hkv, d), dtype),
         "kp": _normal(gen, (case["prefix"], hkv, d), dtype), "vp": _normal(gen, (case["prefix"], hkv, d), dtype)}
    if case["op"] == "train":
        s["dout"] = _normal(gen, (pq[-1], hq, d), dtype)
    return s


def run(s):
    case = s["case"]
    if own:
        import bwd_packed_varlen_gb300 as ta
        if case["op"] == "rope":
            return ta.rope(s["q"], s["k"], s["freq"], s["cu"], s["cu_pad"], start_positions=s["start"], interleaved=case["interleaved"],
                           mscale=s["mscale"], inverse=case["back"])
        cu = (s["cu_q"], s["cu_k"], s["cu_q_pad"], s["cu_k_pad"])
        out, lse = ta.prefix_fwd(s["q"], s["k"], s["v"], s["kp"], s["vp"], *cu, s["scale"], case["mask"])
        if case["op"] == "attend":
            return out, lse
        grads = ta.prefix_bwd(s["q"], s["k"], s["v"], s["kp"], s["vp"], out, s["dout"], lse, *cu, s["scale"], case["mask"])
        return (out, lse) + tuple(grads)
    return _plain_rope(s) if case["op"] == "rope" else _plain_attention(s)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_rope(s):
    case, rot = s["case"], s["case"]["rot"]
    rows = torch.arange(s["q"].shape[0], device="cuda", dtype=torch.int32)
    b = (torch.searchsorted(s["cu_pad"], rows, right=True) - 1).clamp(0, case["batch"] - 1)
    i = rows - s["cu_pad"][b]
    real = i < (s["cu"][1:] - s["cu"][:-1])[b]
    # angles of far positions need 64 bits
    angle = (s["start"][b] + i).double()[:, None] * s["freq"][None, :]
    cos, sin = (angle.cos() * s["mscale"]).float()[:, None, :], (angle.sin() * s["mscale"]).float()[:, None, :]
    if case["back"]:
        sin = -sin

    def turn(x):
        y = x.float()
        if case["interleaved"]:
            a, c = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack((a * cos - c * sin, c * cos + a * sin), dim=-1).flatten(-2)
        else:
            a, c = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat((a * cos - c * sin, c * cos + a * sin), dim=-1)
        z = torch.cat((z, y[..., rot:]), dim=-1)
        return torch.where(real[:, None, None], z, torch.zeros((), device="cuda")).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _rows(cu, cu_pad, longest):
    """Tensor rows of every sequence's tokens as a [batch, longest] table, and which of its places are real."""
    i = torch.arange(longest, device="cuda")
    real = i[None, :] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(real, cu_pad[:-1, None] + i[None, :], 0).long(), real


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d, batch, n_pre = case["hq"], case["hkv"], case["d"], case["batch"], case["prefix"]
    group, nq, nk = hq // hkv, max(s["lq"]), max(s["lk"])
    iq, real_q = _rows(s["cu_q"], s["cu_q_pad"], nq)
    ik, real_k = _rows(s["cu_k"], s["cu_k_pad"], nk)

    def by_head(x, rows):  # [batch, hkv, queries x group, d]
        return x[rows].float().view(batch, nq, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, nq * group, d)

    q = by_head(s["q"], iq)
    k, v = (s[n][ik].float().permute(0, 2, 1, 3) for n in ("k", "v"))  # [batch, hkv, nk, d]
    kp, vp = (s[n].float().permute(1, 0, 2)[None] for n in ("kp", "vp"))  # [1, hkv, prefix, d]
    k, v = (torch.where(real_k[:, None, :, None], x, 0.0) for x in (k, v))
    see = real_q[:, :, None] & real_k[:, None, :]
    if case["mask"] != "padding":
        edge = torch.arange(nq, device="cuda")[None, :, None].expand(batch, nq, 1)
        if case["mask"] == "padding_causal_bottom_right":
            lens = [(c[1:] - c[:-1])[:, None, None] for c in (s["cu_q"], s["cu_k"])]
            edge = edge + lens[1] - lens[0]
        see = see & (torch.arange(nk, device="cuda")[None, None, :] <= edge)
    see = torch.cat((real_q[:, :, None].expand(batch, nq, n_pre), see), dim=-1)
    see = see[:, None, :, None, :].expand(batch, 1, nq, group, n_pre + nk).reshape(batch, 1, nq * group, n_pre + nk)

    def against(x, shared, single):  # x times the prefix's rows, then the sequence's own
        together = x.transpose(0, 1).reshape(1, hkv, batch * nq * group, d) @ shared.transpose(-1, -2)
        return torch.cat((together.view(hkv, batch, nq * group, n_pre).transpose(0, 1), x @ single.transpose(-1, -2)), dim=-1)

    def gather(p, shared, single):
        together = p[..., :n_pre].transpose(0, 1).reshape(1, hkv, batch * nq * group, n_pre) @ shared
        return together.view(hkv, batch, nq * group, d).transpose(0, 1) + p[..., n_pre:] @ single

    score = torch.where(see, against(q, kp, k) * s["scale"], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    del score
    total = p.sum(dim=-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    o = gather(p, vp, v)
    lse = (top + torch.log(total))[..., 0]

    def whole(x, like, rows, real):
        y = torch.zeros_like(like)
        y[rows[real]] = x[real].to(like.dtype)
        return y

    def tokens(x):  # back to [batch, queries, hq, ...]
        return x.view((batch, hkv, nq, group) + x.shape[3:]).transpose(1, 2).flatten(2, 3)

    out = whole(tokens(o), s["q"], iq, real_q)
    lse = whole(tokens(lse), torch.zeros(s["q"].shape[:2], device="cuda"), iq, real_q)
    if case["op"] == "attend":
        return out, lse
    g = by_head(s["dout"], iq) * real_q[:, None, :, None].expand(batch, 1, nq, group).reshape(batch, 1, nq * group, 1)
    dv = p[..., n_pre:].transpose(-1, -2) @ g
    dvp = (p[..., :n_pre].transpose(-1, -2) @ g).sum(0)
    ds = p * (against(g, vp, v) - (g * o).sum(dim=-1, keepdim=True)) * s["scale"]
    del p
    dq = gather(ds, kp, k)
    dk = ds[..., n_pre:].transpose(-1, -2) @ q
    dkp = (ds[..., :n_pre].transpose(-1, -2) @ q).sum(0)
    dk, dv = (whole(x.transpose(1, 2), s["k"], ik, real_k) for x in (dk, dv))
    dkp, dvp = (x.transpose(0, 1).to(s["kp"].dtype) for x in (dkp, dvp))
    return out, lse, whole(tokens(dq), s["q"], iq, real_q), dk, dv, dkp, dvp


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_attention(s)


def _exact_rope(s):
    case, rot = s["case"], s["case"]["rot"]
    pad, start = s["cu_pad"].tolist(), s["start"].tolist()
    outs = []
    for x in (s["q"], s["k"]):
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lengths"]):
            rows = slice(pad[b], pad[b] + n)
            z = x[rows].double()
            y[rows] = z
            pair = z[..., :rot].unflatten(-1, (-1, 2)) if case["interleaved"] else z[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
            pos = torch.arange(start[b], start[b] + n, device="cuda", dtype=torch.float64)
            turned = torch.view_as_complex(pair.contiguous()) * torch.polar(
                torch.full((n, 1, rot // 2), s["mscale"], dtype=torch.float64, device="cuda"),
                (pos[:, None] * s["freq"])[:, None, :] * (-1 if case["back"] else 1))
            pair = torch.view_as_real(turned)
            y[rows, :, :rot] = pair.flatten(-2) if case["interleaved"] else pair.transpose(-1, -2).flatten(-2)
        outs.append(y)
    return tuple(outs)


def _exact_attention(s):
    case = s["case"]
    hq, hkv, d, n_pre = case["hq"], case["hkv"], case["d"], case["prefix"]
    train = case["op"] == "train"
    kp, vp = s["kp"].double().permute(1, 2, 0).contiguous(), s["vp"].double().transpose(0, 1).contiguous()
    zeros = {n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in ("q", "k", "v", "kp", "vp") if train or n == "q"}
    out, lse = torch.zeros_like(zeros["q"]), torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(s["lq"], s["lk"])):
        if n == 0:
            continue
        rq, rk = slice(s["pq"][b], s["pq"][b] + n), slice(s["pk"][b], s["pk"][b] + m)
        leaves = [s["q"][rq].double(), s["k"][rk].double(), s["v"][rk].double(), kp, vp]
        if train:
            leaves = [x.detach().requires_grad_() for x in leaves]
        q, k, v, kq, vq = leaves
        q4 = q.view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
        blocked = torch.zeros(n, n_pre + m, dtype=torch.bool, device="cuda")
        if case["mask"] != "padding":
            shift = m - n if case["mask"] == "padding_causal_bottom_right" else 0
            blocked[:, n_pre:] = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(1 + shift)
        score = torch.cat((torch.matmul(q4, kq), torch.matmul(q4, k.permute(1, 2, 0))), dim=-1) * s["scale"]
        score = score.view(hkv, hq // hkv, n, n_pre + m).masked_fill(blocked, -math.inf)
        p = torch.softmax(score, dim=-1).view(hkv, -1, n_pre + m)
        o = (torch.matmul(p[..., :n_pre], vq) + torch.matmul(p[..., n_pre:], v.transpose(0, 1))).view(hq, n, d).transpose(0, 1)
        out[rq] = o.detach()
        lse[rq] = torch.logsumexp(score.detach(), dim=-1).reshape(hq, n).t()
        if train:
            got = torch.autograd.grad(o, leaves, s["dout"][rq].double())
            for name, rows, x in zip(("q", "k", "v"), (rq, rk, rk), got):
                zeros[name][rows] = x
            zeros["kp"] += got[3].permute(2, 0, 1)
            zeros["vp"] += got[4].transpose(0, 1)
    return (out, lse) + (tuple(zeros[n] for n in ("q", "k", "v", "kp", "vp")) if train else ())
