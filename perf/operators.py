"""Paged K / V cache operators, measured: writing (and quantising) new tokens, reading them back, and
attention of a chunk of new tokens over the cache.

A case names its sizes; ``prepare`` makes the inputs, ``run`` is one pass (plain torch where ``own`` is
false, the library's call where it is true), ``exact`` the same in 64 bits, ``work`` the bytes and
operations a pass cannot do without.

The cache holds pages of ``page`` tokens, [pages, kv heads, page, D], as bf16, e4m3 or int8; the 8-bit
formats carry one power-of-two scale (a biased exponent byte) for every 32 channels of a token.  Token i
of the n that cu_seq gives sequence s stands at position kv_len[s] - n + i of that sequence.
"""
import math
import random

import torch

own = False

GROUP = 32            # channels under one scale
LEAST_EXPONENT = -117  # of a scale: e4m3's smallest step times it is bf16's smallest normal number
FORMATS = ("bf16", "fp8", "int8")


# ----------------------------------------------------------------------------------------- cases --
def listed():
    return [
        # one decode step of a served batch: a token for each of 32 sequences, small pages
        dict(name="write-step-int8", op="write", seqs=32, n_lo=1, n_hi=1, ctx=4000, kv_heads=8, dim=128, page=16,
             format="int8", head_major=False),
        # a few requests of odd lengths in the [H, T, D] layout that the attention layer keeps
        dict(name="write-ragged-bf16", op="write", seqs=5, n_lo=1, n_hi=701, ctx=900, kv_heads=10, dim=64, page=32,
             format="bf16", head_major=True),
        # one latent frame of the 1.3B-like 480p layer (30 x 52 tokens, 12 heads) appended to a video's cache
        dict(name="write-frame-fp8", op="write", seqs=1, n_lo=1560, n_hi=1560, ctx=7800, kv_heads=12, dim=128,
             page=64, format="fp8", head_major=False),
        # all 21 frames of the 14B-like 480p layer (40 heads) at once: the prompt of a continuation
        dict(name="write-video-fp8", op="write", seqs=1, n_lo=32760, n_hi=32760, ctx=0, kv_heads=40, dim=128, page=64,
             format="fp8", head_major=False),
        # the last tokens of a few sequences fetched back
        dict(name="read-tails-int8", op="read", seqs=3, n_lo=1, n_hi=257, ctx=2000, kv_heads=2, dim=64, page=16,
             format="int8", head_major=False),
        # a 480p video's whole history as the [H, N, D] tensor that the block-sparse layer takes
        dict(name="read-history-fp8", op="read", seqs=1, n_lo=32760, n_hi=32760, ctx=0, kv_heads=40, dim=128, page=64,
             format="fp8", head_major=True),
        # one token of one sequence: the call's latency
        dict(name="attend-one-bf16", op="attend", seqs=1, n_lo=1, n_hi=1, ctx=776, heads=12, kv_heads=12, dim=128,
             page=16, format="bf16", frame=1, window=0),
        # a served batch's decode step, lengths far apart, four query heads to a K / V head
        dict(name="attend-batch-int8", op="attend", seqs=64, n_lo=1, n_hi=1, ctx=16000, heads=32, kv_heads=8, dim=128,
             page=16, format="int8", frame=1, window=0),
        # single tokens over very long caches: all of the time is reading them
        dict(name="attend-long-fp8", op="attend", seqs=3, n_lo=1, n_hi=1, ctx=-131071, heads=64, kv_heads=8, dim=128,
             page=64, format="fp8", frame=1, window=0),
        # prompts' next chunks beside single tokens in one call; five query heads to a K / V head
        dict(name="attend-ragged-bf16", op="attend", seqs=8, n_lo=1, n_hi=1024, ctx=3000, heads=40, kv_heads=8, dim=64,
             page=32, format="bf16", frame=1, window=0),
        # one frame of the 1.3B-like 480p layer over its video so far, causal by frames, the last 12 frames seen
        dict(name="attend-frame-bf16", op="attend", seqs=1, n_lo=1560, n_hi=1560, ctx=-31200, heads=12, kv_heads=12,
             dim=128, page=64, format="bf16", frame=1560, window=12),
        # the same of the 14B-like layer (40 heads) over the whole video, kept in e4m3
        dict(name="attend-frame-fp8", op="attend", seqs=1, n_lo=1560, n_hi=1560, ctx=-31200, heads=40, kv_heads=40,
             dim=128, page=64, format="fp8", frame=1560, window=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend"))
    dim, page, fmt = rng.choice((64, 128, 128)), rng.choice((16, 32, 64, 128)), rng.choice(FORMATS)
    while True:
        seqs = _log_int(rng, 1, 64)
        n_hi = _log_int(rng, 1, 32760)
        n_lo = rng.choice((1, n_hi, max(1, n_hi // 3)))
        kv_heads = rng.choice((1, 2, 5, 8, 12, 24, 40))
        c = dict(op=op, seqs=seqs, n_lo=n_lo, n_hi=n_hi, kv_heads=kv_heads, dim=dim, page=page, format=fmt)
        if op != "attend":
            c.update(ctx=rng.choice((0, _log_int(rng, 1, 8000))), head_major=rng.random() < 0.5)
            if seqs * (c["ctx"] + n_hi) * kv_heads * dim <= 32760 * 40 * 128:
                return c
            continue
        group = rng.choice((1, 1, 2, 4, 5, 8))
        frame = rng.choice((0, 1, 1, 16, 1560))
        c.update(n_hi=1 if rng.random() < 0.4 else min(n_hi, 8192), ctx=_log_int(rng, 1, 131071),
                 heads=kv_heads * group, frame=frame,
                 window=0 if frame == 0 or rng.random() < 0.6 else _log_int(rng, 1, 16 if frame > 1 else 4096))
        c["n_lo"] = min(n_lo, c["n_hi"])
        keys = c["ctx"] + c["n_hi"]
        # the plain form keeps every score of the padded batch
        if seqs * c["heads"] * c["n_hi"] * keys <= 40 * 1560 * 32760 and seqs * keys * kv_heads * dim <= 3 * 131072 * 8 * 128:
            return c


def _lengths(case):
    """(new tokens, length with them) of each sequence: a part of the case.  ctx < 0: every sequence has -ctx."""
    rng = random.Random("%s-%s-%s-%s" % (case["seqs"], case["n_lo"], case["n_hi"], case["ctx"]))
    ns, lens = [], []
    for s in range(case["seqs"]):
        n = case["n_hi"] if s == 0 else rng.randint(case["n_lo"], case["n_hi"])
        ctx = -case["ctx"] if case["ctx"] < 0 else case["ctx"] if s == 0 else rng.randint(0, case["ctx"])
        ns.append(n)
        lens.append(ctx + n)
    return ns, lens


def _bounds(case, length, n, i):
    """Positions [lo, hi) that token i of n sees."""
    if case["frame"] == 0:
        return 0, length
    f = (length - n + i) // case["frame"]
    return (max(0, (f - case["window"] + 1) * case["frame"]) if case["window"] else 0), min(length, (f + 1) * case["frame"])


def work(case):
    ns, lens = _lengths(case)
    d, hk = case["dim"], case["kv_heads"]
    token = 2 * hk * (2 * d if case["format"] == "bf16" else d + d // GROUP)  # K and V of one cached token
    if case["op"] != "attend":
        t = sum(ns)
        return {"bytes": t * (token + 2 * hk * d * 2), "flops": 0 if case["format"] == "bf16" else 4 * t * hk * d}
    keys = pairs = 0
    for n, length in zip(ns, lens):
        seen = [_bounds(case, length, n, i) for i in range(n)]
        keys += max(h for _, h in seen) - min(lo for lo, _ in seen)
        pairs += sum(h - lo for lo, h in seen)
    rows = sum(ns) * case["heads"]
    return {"bytes": keys * token + rows * (d * 4 + 4), "flops": 4 * d * case["heads"] * pairs}


# ---------------------------------------------------------------------------------------- inputs --
def _quantise(x, fmt):
    """bf16 [..., D] -> (stored values, exponent bytes [..., D / 32] or None)."""
    if fmt == "bf16":
        return x, None
    g = x.float().unflatten(-1, (-1, GROUP))
    frac, ex = torch.frexp(g.abs().amax(-1))
    # least e with amax <= 448 * 2^e (448 = 0.875 * 2^9) or <= 127 * 2^e (127 = 0.9921875 * 2^7)
    top, bits = (0.875, 9) if fmt == "fp8" else (0.9921875, 7)
    e = torch.where(frac <= top, ex - bits, ex - bits + 1).clamp(min=LEAST_EXPONENT)
    y = torch.ldexp(g, -e.unsqueeze(-1)).flatten(-2)
    y = y.to(torch.float8_e4m3fn) if fmt == "fp8" else y.round().to(torch.int8)
    return y, (e + 127).to(torch.uint8)


def _values(x, scale, dtype=torch.float32):
    """Stored values -> what they stand for."""
    if scale is None:
        return x.to(dtype)
    e = scale.to(torch.int32) - 127
    return torch.ldexp(x.to(dtype).unflatten(-1, (-1, GROUP)), e.unsqueeze(-1)).flatten(-2)


def _kv(shape, gen, dev):
    """Keys or values: unit noise, a part that the tokens share, and a few strong channels."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    gain = 1.0 + 3.0 * (torch.rand(shape[-1], generator=gen, device=dev) < 0.06)
    shared = 0.7 * torch.randn(shape[-1], generator=gen, device=dev)
    return ((x + shared.bfloat16()) * gain.bfloat16())


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(seed)
    ns, lens = _lengths(case)
    page, hk, d, fmt = case["page"], case["kv_heads"], case["dim"], case["format"]
    used = [-(-n // page) for n in lens]
    cols, pages = max(used), sum(used) + 3   # three pages belong to nobody
    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int32)
    starts = torch.tensor([sum(used[:s]) for s in range(len(used))], device=dev)
    col = torch.arange(cols, device=dev)
    # entries behind a sequence's last page are other sequences' pages, never to be looked at
    table = order[(starts[:, None] + col[None]) % pages].contiguous()
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    st = dict(case=case, table=table, cu=torch.tensor(cu, device=dev, dtype=torch.int32),
              length=torch.tensor(lens, device=dev, dtype=torch.int32), tokens=cu[-1], most=max(ns), longest=max(lens))
    # for the plain form: the sequence of each token and its number in it
    seq = torch.repeat_interleave(torch.arange(len(ns), device=dev), torch.tensor(ns, device=dev))
    st["seq"], st["off"] = seq, torch.arange(cu[-1], device=dev) - st["cu"][seq]
    shape = (pages, hk, page, d)
    if case["op"] == "write":
        kind = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[fmt]
        st["k"], st["v"] = (torch.zeros(shape, device=dev).to(kind) for _ in range(2))
        st["ks"], st["vs"] = (None if fmt == "bf16" else torch.full(shape[:3] + (d // GROUP,), 127, device=dev,
                                                                    dtype=torch.uint8) for _ in range(2))
        new = (hk, cu[-1], d) if case["head_major"] else (cu[-1], hk, d)
        st["new_k"], st["new_v"] = (_kv(new, gen, dev) for _ in range(2))
        if case["head_major"]:
            st["new_k"], st["new_v"] = st["new_k"].transpose(0, 1), st["new_v"].transpose(0, 1)
    else:
        (st["k"], st["ks"]), (st["v"], st["vs"]) = (_quantise(_kv(shape, gen, dev), fmt) for _ in range(2))
    if case["op"] == "attend":
        st["q"] = torch.randn((cu[-1], case["heads"], d), generator=gen, device=dev, dtype=torch.bfloat16)
    return st


# ------------------------------------------------------------------------------------ plain forms --
def _places(st):
    """(page, slot) of each token."""
    c = st["case"]
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    pos = st["length"].long()[st["seq"]] - n[st["seq"]] + st["off"]
    return st["table"][st["seq"], pos // c["page"]].long(), pos % c["page"]


def _write(st):
    page, slot = _places(st)
    for new, held, scale in (("new_k", "k", "ks"), ("new_v", "v", "vs")):
        y, e = _quantise(st[new], st["case"]["format"])
        raw = torch.int16 if e is None else torch.uint8   # an indexed copy of the stored bits
        st[held].view(raw)[page, :, slot] = y.contiguous().view(raw)
        if e is not None:
            st[scale][page, :, slot] = e
    return st["k"], st["v"], st["ks"], st["vs"]


def _read(st):
    page, slot = _places(st)
    out = []
    for held, scale in (("k", "ks"), ("v", "vs")):
        raw = torch.int16 if st[scale] is None else torch.uint8
        x = st[held].view(raw)[page, :, slot].view(st[held].dtype)
        x = _values(x, None if st[scale] is None else st[scale][page, :, slot]).to(torch.bfloat16)
        out.append(x.transpose(0, 1).contiguous() if st["case"]["head_major"] else x)
    return tuple(out)


def _attend(st):
    c = st["case"]
    hk, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    seqs, most = c["seqs"], st["most"]
    n, length = (st["cu"][1:] - st["cu"][:-1]).long(), st["length"].long()
    pages = st["table"].long()
    keys = pages.shape[1] * c["page"]

    def all_keys(held, scale):
        raw = torch.int16 if st[scale] is None else torch.uint8
        x = st[held].view(raw)[pages].view(st[held].dtype)
        x = _values(x, None if st[scale] is None else st[scale][pages])
        return x.transpose(1, 2).reshape(seqs, hk, keys, d)

    i = torch.arange(most, device=n.device)
    at = (st["cu"][:-1].long()[:, None] + i[None]).clamp(max=st["tokens"] - 1)
    q = st["q"][at].float().unflatten(2, (hk, g)).permute(0, 2, 3, 1, 4).reshape(seqs, hk, g * most, d)
    s = torch.matmul(q, all_keys("k", "ks").transpose(2, 3)) * (1.0 / math.sqrt(d))
    pos = (length - n)[:, None] + i[None]
    lo, hi = torch.zeros_like(pos), length[:, None].expand_as(pos)
    if c["frame"]:
        f = torch.div(pos, c["frame"], rounding_mode="floor")
        hi = torch.minimum(hi, (f + 1) * c["frame"])
        if c["window"]:
            lo = ((f - c["window"] + 1) * c["frame"]).clamp(min=0)
    key = torch.arange(keys, device=n.device)
    seen = ((key >= lo[..., None]) & (key < hi[..., None]))[:, None, None]
    s = s.view(seqs, hk, g, most, keys).masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hk, g * most, keys), all_keys("v", "vs")).view(seqs, hk, g, most, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, most, c["heads"], d)[st["seq"], st["off"]]
    lse = lse.permute(0, 3, 1, 2).reshape(seqs, most, c["heads"])[st["seq"], st["off"]]
    return o.to(torch.bfloat16), lse.transpose(0, 1).contiguous()


def run(st):
    c = st["case"]
    if own:
        from block_sparse_attention_candidate_b200 import abi
        cache = abi.KVCache(st["k"], st["v"], st["ks"], st["vs"])
        if c["op"] == "write":
            abi.dynrad_cache_write(cache, st["new_k"], st["new_v"], st["table"], st["cu"], st["length"])
            return st["k"], st["v"], st["ks"], st["vs"]
        if c["op"] == "read":
            return abi.dynrad_cache_read(cache, st["table"], st["cu"], st["length"], st["tokens"],
                                         head_major=c["head_major"])
        return abi.dynrad_cache_attn(st["q"], cache, st["table"], st["cu"], st["length"], frame=c["frame"],
                                     window=c["window"])
    return {"write": _write, "read": _read, "attend": _attend}[c["op"]](st)


# ------------------------------------------------------------------------------------------ exact --
def _exact_stored(x, fmt):
    """The definition in 64 bits, for e4m3: per 32 channels the least power of two that brings them
    within the format's range, and each channel's nearest step there (ties to even)."""
    if fmt == "bf16":
        return x.double()
    limit = 448.0
    x = x.double().unflatten(-1, (-1, GROUP))
    most = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.clamp(most, min=1e-300) / limit))
    e = torch.where(most > limit * torch.exp2(e), e + 1, e)
    e = torch.where(most <= limit * torch.exp2(e - 1), e - 1, e).clamp(min=LEAST_EXPONENT)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -6))) - 3)  # 3 bits, least exponent -6
    return (torch.round(y / step) * step).flatten(-2)


def _exact_kept(x, scale):
    x = x.double()
    if scale is None:
        return x
    return x * torch.exp2(scale.double() - 127).repeat_interleave(GROUP, -1)


def exact(case, seed):
    st = prepare(case, seed)
    ns, lens = _lengths(case)
    table, page = st["table"].tolist(), case["page"]
    where, base = [], 0
    for s, (n, length) in enumerate(zip(ns, lens)):
        where.append((base, n, length, torch.tensor(table[s], device="cuda")))
        base += n
    if case["op"] == "write":
        fmt, out = case["format"], []
        if fmt == "int8":
            return None  # whole numbers alone: they have to equal the plain form's
        for new, held in (("new_k", "k"), ("new_v", "v")):
            y = _exact_stored(st[new], fmt)
            to = st[held].double()
            for base, n, length, pages in where:
                at = torch.arange(length - n, length, device="cuda")
                to[pages[at // page], :, at % page] = y[base:base + n]
            out.append(to)
        return out + [None, None]
    if case["op"] == "read":
        out = []
        for held, scale in (("k", "ks"), ("v", "vs")):
            rows = []
            for base, n, length, pages in where:
                at = torch.arange(length - n, length, device="cuda")
                raw = st[held].view(torch.int16 if st[scale] is None else torch.uint8)[pages[at // page], :, at % page]
                rows.append(_exact_kept(raw.view(st[held].dtype), None if st[scale] is None
                                        else st[scale][pages[at // page], :, at % page]))
            x = torch.cat(rows)
            out.append(x.transpose(0, 1).contiguous() if case["head_major"] else x)
        return out
    g, d = case["heads"] // case["kv_heads"], case["dim"]
    o = torch.zeros((st["tokens"], case["heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((case["heads"], st["tokens"]), -math.inf, dtype=torch.float64, device="cuda")
    for base, n, length, pages in where:
        span = [_bounds(case, length, n, i) for i in range(n)]
        lo, hi = (torch.tensor(x, device="cuda")[:, None] for x in zip(*span))
        key = torch.arange(length, device="cuda")
        seen = (key >= lo) & (key < hi)
        use = pages[:-(-length // page)]
        for h in range(case["kv_heads"]):
            k, v = (_exact_kept(st[a][use, h], None if st[b] is None else st[b][use, h]).reshape(-1, d)[:length]
                    for a, b in (("k", "ks"), ("v", "vs")))
            for r in range(g):
                logits = st["q"][base:base + n, h * g + r].double() @ k.T / math.sqrt(d)
                logits = logits.masked_fill(~seen, -math.inf)
                z = torch.logsumexp(logits, -1)
                w = torch.exp(logits - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
                o[base:base + n, h * g + r] = w @ v
                lse[h * g + r, base:base + n] = z
    return o, lse
