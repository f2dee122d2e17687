"""Paged K / V cache on the GPU against the float64 oracle: stored codes and
scales and the read-back exactly, attention within bounds by arithmetic."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_candidate_b200 import abi
from cache_util import (Batch, DTYPE, check_attention, empty_cache, f64, filled_cache)
from gpu_util import check_device_status, full_csr
from oracle import cache as OC

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "fp8", "int8"]


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def odd_values(shape, seed):
    """bf16 with magnitudes over the whole range, zeros, subnormals, exact powers
    of two and borders of the formats, and groups that hold an infinity or a NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    flat = x.view(-1, 32)
    n = flat.shape[0]
    e = torch.randint(-130, 126, (n, 1), generator=g).double()
    e[::3] = 0
    flat = (flat.double() * torch.exp2(e)).float().clamp(-3.0e38, 3.0e38)
    flat[1::17] = 0.0
    flat[2::17, 5] = -0.0
    flat[3::17, 0] = 448.0
    flat[3::17, 1:] = flat[3::17, 1:].clamp(-440, 440)
    flat[4::17] = torch.arange(32).float() * 13.9375 * (1 - 2 * (torch.arange(32) % 2))
    flat[5::17, 3] = 127.0
    flat[5::17, 4:] = torch.arange(28) + 0.5
    flat[6::17, 0] = 127.5
    flat[7::17, 31] = math.inf
    flat[8::17, 0] = math.nan
    flat[9::17, 2] = -math.inf
    flat[10::17] = 1e-39
    flat[11::17, 1] = 3.3895e38
    return flat.view(shape).bfloat16()


def laid_out(x, layout):
    """The same values as [T, H, D], as a transposed [H, T, D], or inside a wider tensor."""
    if layout == "thd":
        return x.contiguous()
    if layout == "htd":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((x.shape[0], x.shape[1] + 1, x.shape[2] + 8), math.nan, dtype=x.dtype, device=x.device)
    wide[:, :-1, 8:] = x
    return wide[:, :-1, 8:]


WRITE_BATCHES = [([1], [1]), ([1, 0, 5], [7, 3, 5]), ([33, 1, 64], [50, 129, 64]), ([3, 9], [2, 9])]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,layout", [(16, "thd"), (32, "htd"), (64, "wide"), (128, "thd")])
@pytest.mark.parametrize("which", range(len(WRITE_BATCHES)))
def test_write_stores_the_oracles_codes_and_nothing_else(fmt, dim, page, layout, which):
    ns, lens = WRITE_BATCHES[which]
    b = Batch(ns, lens, page, seed=which, tail=which % 2 * 3)
    heads = 3
    x = {n: odd_values((b.tokens, heads, dim), 10 * which + i).cuda() for i, n in enumerate("kv")}
    c = empty_cache(b, heads, dim, fmt)
    abi.dynrad_cache_write(c, laid_out(x["k"], layout), laid_out(x["v"], layout), *b.call())
    torch.cuda.synchronize()
    check_device_status()
    raw = torch.int16 if fmt == "bf16" else torch.uint8
    for name, held, scale in (("k", c.k, c.k_scale), ("v", c.v, c.v_scale)):
        want = np.full(held.shape, -1 if fmt == "bf16" else 255, dtype=np.int16 if fmt == "bf16" else np.uint8)
        wscale = None if scale is None else np.full(scale.shape, 255, dtype=np.uint8)
        bits = x[name].view(torch.int16).cpu().numpy()
        code, byte = (bits, None) if fmt == "bf16" else OC.quantise(f64(x[name]), fmt)
        for s, (n, length) in enumerate(zip(ns, lens)):
            for i in range(n):
                pos = length - n + i
                if pos < 0:
                    continue
                pg, slot = OC.place(b.table_np, page, s, pos)
                want[pg, :, slot] = code[b.cu_np[s] + i]
                if byte is not None:
                    wscale[pg, :, slot] = byte[b.cu_np[s] + i]
        assert np.array_equal(held.view(raw).cpu().numpy(), want)
        if byte is not None:
            assert np.array_equal(scale.cpu().numpy(), wscale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,head_major", [(16, False), (32, True), (64, False), (128, True)])
def test_read_back_is_exactly_what_is_stored(fmt, dim, page, head_major):
    b = Batch([5, 0, 40, 3], [70, 9, 40, 2], page, seed=3, tail=2)
    heads, w = 2, b.whole()
    x = {n: odd_values((w.tokens, heads, dim), 50 + i).cuda() for i, n in enumerate("kv")}
    c = empty_cache(b, heads, dim, fmt)
    abi.dynrad_cache_write(c, x["k"], x["v"], *w.call())
    shape = (heads, b.tokens, dim) if head_major else (b.tokens, heads, dim)
    out = tuple(torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    abi.dynrad_cache_read(c, *b.call(), head_major=head_major, out=out)
    torch.cuda.synchronize()
    check_device_status()
    for name, o in zip("kv", out):
        o = (o.transpose(0, 1) if head_major else o).float().cpu().numpy()
        kept = f64(x[name])
        if fmt != "bf16":
            kept = OC.stands_for(*OC.quantise(kept, fmt), fmt)
        for s, (n, length) in enumerate(zip(b.ns, b.lens)):
            for i in range(n):
                pos = length - n + i
                want = np.zeros((heads, dim)) if pos < 0 else kept[w.cu_np[s] + pos]
                got = o[b.cu_np[s] + i].astype(np.float64)
                assert np.array_equal(got, want, equal_nan=True), (name, s, i)
        assert (o[b.cu_np[-1]:] == 7.0).all()      # rows that belong to nobody


# (new tokens, lengths): single tokens, chunks from nothing, odd sizes, a sequence
# without tokens, one without keys, one with more tokens than positions
BATCHES = {
    "one": ([1], [1]),
    "token": ([1, 1, 1], [1, 300, 127]),
    "prompt": ([130], [130]),
    "mixed": ([1, 37, 0, 129, 1], [513, 40, 77, 400, 0]),
    "short": ([5, 260], [3, 257]),
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("heads,kv_heads,page,frame,window", [
    (2, 2, 16, 1, 0), (6, 2, 32, 1, 40), (5, 1, 64, 0, 0), (8, 1, 128, 24, 3)])
@pytest.mark.parametrize("cut", [False, True])
def test_attention_matches_the_oracle(fmt, dim, name, heads, kv_heads, page, frame, window, cut):
    ns, lens = BATCHES[name]
    b = Batch(ns, lens, page, seed=len(name), tail=3, keys=1100 if cut else 0, skip=2)
    g = gen(dim + len(name))
    c, kk, kv = filled_cache(b, kv_heads, dim, fmt, g)
    q = torch.randn((b.tokens, heads, dim), generator=g, device="cuda").bfloat16()
    o = torch.full_like(q, 7.0)
    lse = torch.full((heads, b.tokens), 7.0, device="cuda")
    abi.dynrad_cache_attn(q, c, *b.call(), frame=frame, window=window, out=o, lse=lse)
    torch.cuda.synchronize()
    check_device_status()
    check_attention(o, lse, q, kk, kv, b, frame, window)
    for nobodys in (slice(0, 2), slice(int(b.cu_np[-1]), None)):
        assert (o[nobodys] == 7.0).all() and (lse[:, nobodys] == 7.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ns,lens,heads,kv_heads,dim,page,frame,window", [
    ([1], [9000], 4, 1, 128, 16, 1, 0),                      # one item cut into many parts
    ([1, 1, 1], [5000, 1, 2600], 8, 2, 64, 32, 1, 700),
    ([2, 600], [4000, 1500], 2, 2, 128, 64, 1, 0),           # two tiles an item, parts of both
    ([300], [2500], 10, 2, 64, 128, 100, 4),
    ([257, 1, 255], [700, 900, 255], 3, 3, 128, 32, 0, 0),
])
def test_items_cut_into_parts(fmt, ns, lens, heads, kv_heads, dim, page, frame, window):
    b = Batch(ns, lens, page, seed=len(lens))
    g = gen(page + heads)
    c, kk, kv = filled_cache(b, kv_heads, dim, fmt, g)
    q = torch.randn((b.tokens, heads, dim), generator=g, device="cuda").bfloat16()
    o, lse = abi.dynrad_cache_attn(q, c, *b.call(), frame=frame, window=window)
    torch.cuda.synchronize()
    check_device_status()
    check_attention(o, lse, q, kk, kv, b, frame, window)
    o2, lse2 = abi.dynrad_cache_attn(q, c, *b.call(), frame=frame, window=window)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("ns,lens,heads,kv_heads", [
    ([1700], [1750], 192, 12),              # items in many waves: one to a CTA
    ([900, 1, 830, 0, 60], [950, 70, 830, 5, 300], 192, 12),
    ([1] * 2100, [1 + i % 37 for i in range(2100)], 2, 1),      # more places than a CTA scans
])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_calls_of_many_items(ns, lens, heads, kv_heads, fmt):
    b = Batch(ns, lens, 32, seed=1, keys=1100)
    g = gen(len(ns))
    c, kk, kv = filled_cache(b, kv_heads, 64, fmt, g)
    q = torch.randn((b.tokens, heads, 64), generator=g, device="cuda").bfloat16()
    o, lse = abi.dynrad_cache_attn(q, c, *b.call())
    torch.cuda.synchronize()
    check_device_status()
    check_attention(o, lse, q, kk, kv, b, 1, 0)


def test_a_wait_that_runs_out_is_recorded_and_the_next_call_is_right():
    b = Batch([1, 200], [800, 700], 64, seed=3)
    g = gen(6)
    for fmt in FORMATS:
        c, kk, kv = filled_cache(b, 2, 128, fmt, g)
        q = torch.randn((b.tokens, 4, 128), generator=g, device="cuda").bfloat16()
        check_device_status()
        abi.dynrad_debug_attn_stall(20_000, 1)
        try:
            abi.dynrad_cache_attn(q, c, *b.call())
            torch.cuda.synchronize()
        finally:
            abi.dynrad_debug_attn_stall()
        assert abi.dynrad_device_status(clear=True) == abi.DYNRAD_ERR_DEVICE
        o, lse = abi.dynrad_cache_attn(q, c, *b.call())
        torch.cuda.synchronize()
        check_device_status()
        check_attention(o, lse, q, kk, kv, b, 1, 0)


@pytest.mark.parametrize("heads,kv_heads", [(7, 1), (12, 4), (40, 8), (128, 1), (3, 3)])
def test_head_groups_and_layouts(heads, kv_heads):
    b = Batch([3, 150, 1], [200, 150, 90], 32, seed=5)
    g = gen(heads)
    c, kk, kv = filled_cache(b, kv_heads, 64, "fp8", g)
    q = torch.randn((b.tokens, heads, 64), generator=g, device="cuda").bfloat16()
    o, lse = abi.dynrad_cache_attn(q, c, *b.call())
    check_attention(o, lse, q, kk, kv, b, 1, 0)
    for layout in ("htd", "wide"):
        out = laid_out(torch.zeros_like(q), layout)
        o2, lse2 = abi.dynrad_cache_attn(laid_out(q, layout), c, *b.call(), out=out)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
    check_device_status()


@pytest.mark.parametrize("frame,window", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1), (7, 1), (130, 1)])
def test_extreme_frames_and_windows(frame, window):
    for fmt, ns in (("bf16", [40, 1]), ("fp8", [40, 1]), ("fp8", [1, 2])):
        b = Batch(ns, [290, 131], 16, seed=6, keys=1100)
        g = gen(8)
        c, kk, kv = filled_cache(b, 1, 64, fmt, g)
        q = torch.randn((b.tokens, 3, 64), generator=g, device="cuda").bfloat16()
        o, lse = abi.dynrad_cache_attn(q, c, *b.call(), frame=frame, window=window)
        torch.cuda.synchronize()
        check_device_status()
        check_attention(o, lse, q, kk, kv, b, frame, window)


@pytest.mark.parametrize("scale", [0.02, 0.7])
def test_logit_scale_and_strong_logits(scale):
    b = Batch([1, 70], [260, 200], 64, seed=6)
    g = gen(1)
    c, kk, kv = filled_cache(b, 2, 128, "bf16", g, scale=3.0)
    q = (4.0 * torch.randn((b.tokens, 4, 128), generator=g, device="cuda")).bfloat16()
    o, lse = abi.dynrad_cache_attn(q, c, *b.call(), scale=scale)
    check_device_status()
    check_attention(o, lse, q, kk, kv, b, 1, 0, scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("frame,window", [(1, 0), (1, 20), (16, 2)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("ns,cut", [([100, 1], False), ([100, 1], True), ([2, 3], True)])
def test_what_a_row_does_not_see_cannot_reach_it(fmt, frame, window, bad, ns, cut):
    """A token whose K and V hold NaN or infinity, inside the cache: rows that do
    not see it are those of the finite cache, rows that see it are not finite."""
    b = Batch(ns, [112, 33] if ns == [2, 3] else [150, 140], 32, seed=8, keys=1100 if cut else 0)
    g = gen(3)
    w = b.whole()
    k, v = (torch.randn((w.tokens, 2, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((b.tokens, 4, 64), generator=g, device="cuda").bfloat16()
    clean, _, _ = filled_cache(b, 2, 64, fmt, g, k=k, v=v)
    o_ref, lse_ref = abi.dynrad_cache_attn(q, clean, *b.call(), frame=frame, window=window)
    hit = [110, w.cu_np[1] + 30]                      # a position of each sequence
    k2, v2 = k.clone(), v.clone()
    v2[hit, :, 5] = bad
    dirty, _, _ = filled_cache(b, 2, 64, fmt, g, k=k2, v=v2)
    o, lse = abi.dynrad_cache_attn(q, dirty, *b.call(), frame=frame, window=window)
    torch.cuda.synchronize()
    check_device_status()
    assert torch.equal(lse, lse_ref)                  # K is the same
    for s in range(2):
        for i in range(b.ns[s]):
            lo, hi = OC.seen(frame, window, b.lens[s] - b.ns[s] + i, b.lens[s])
            pos = 110 if s == 0 else 30
            t = int(b.cu_np[s]) + i
            if lo <= pos < hi:
                assert not torch.isfinite(o[t, :, 5]).any()
                group = 1 if fmt == "bf16" else 32       # what shares the bad channel's scale
                assert torch.equal(o[t, :, group if group > 1 else 6:], o_ref[t, :, group if group > 1 else 6:])
                if fmt == "bf16" and math.isinf(bad):
                    assert (o[t, :, 5] == bad).all()
            else:
                assert torch.equal(o[t], o_ref[t]), (s, i)
    # the same in K: a logit that is not a number, for the rows that see it
    k2[hit, :, 5] = math.nan
    dirty, _, _ = filled_cache(b, 2, 64, fmt, g, k=k2, v=v)
    o, lse = abi.dynrad_cache_attn(q, dirty, *b.call(), frame=frame, window=window)
    for s in range(2):
        for i in range(b.ns[s]):
            lo, hi = OC.seen(frame, window, b.lens[s] - b.ns[s] + i, b.lens[s])
            t = int(b.cu_np[s]) + i
            if lo <= (110 if s == 0 else 30) < hi:
                assert torch.isnan(o[t]).all() and torch.isnan(lse[:, t]).all()
            else:
                assert torch.equal(o[t], o_ref[t]) and torch.equal(lse[:, t], lse_ref[:, t])


def test_bad_pages_and_offsets_are_held_and_recorded():
    b = Batch([4, 6], [40, 20], 16, seed=9)
    g = gen(4)
    for what in ("page", "cu", "len"):
        c, kk, kv = filled_cache(b, 1, 64, "int8", g)
        table, cu, length = (t.clone() for t in b.call())
        if what == "page":
            table[0, 1] = b.num_pages
            kk[0][16:32] = 0.0
            kv[0][16:32] = 0.0
        elif what == "cu":
            cu[2] = 1000
        else:
            length[1] = 10 ** 6
        q = torch.randn((b.tokens, 2, 64), generator=g, device="cuda").bfloat16()
        check_device_status()
        o, lse = abi.dynrad_cache_attn(q, c, table, cu, length)
        torch.cuda.synchronize()
        assert abi.dynrad_device_status(clear=True) == abi.DYNRAD_ERR_DEVICE
        if what == "page":
            check_attention(o, lse, q, kk, kv, b, 1, 0)
            k, _ = abi.dynrad_cache_read(c, table, torch.tensor([0, 40, 60], dtype=torch.int32, device="cuda"),
                                         length, 60)
            assert (k[16:32] == 0).all() and (k[:16] != 0).any()
            before = c.k.clone()
            abi.dynrad_cache_write(c, q[:, :1], q[:, :1], table, cu, torch.tensor([20, 20], dtype=torch.int32,
                                                                                  device="cuda"))
            torch.cuda.synchronize()
            assert abi.dynrad_device_status(clear=True) == abi.DYNRAD_ERR_DEVICE
            pg, slot = OC.place(b.table_np, 16, 1, 14)
            same = before.clone()
            for i in range(6):
                pg, slot = OC.place(b.table_np, 16, 1, 14 + i)
                same[pg, :, slot] = c.k[pg, :, slot]
            assert torch.equal(same, c.k)          # the sequence with the bad page wrote nothing


def test_empty_calls():
    b = Batch([0, 0], [5, 0], 16)
    c, _, _ = filled_cache(b, 1, 64, "bf16", gen(0))
    q = torch.ones((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    o, lse = abi.dynrad_cache_attn(q, c, *b.call())
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    abi.dynrad_cache_write(c, q[:, :1], q[:, :1], *b.call())
    k, v = abi.dynrad_cache_read(c, *b.call(), 0)
    assert k.shape == (0, 1, 64)
    none = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    q = torch.full((3, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    out = q.clone()
    abi.dynrad_cache_attn(q, c, none, torch.zeros(1, dtype=torch.int32, device="cuda"), none[:, 0], out=out)
    torch.cuda.synchronize()
    check_device_status()
    assert torch.equal(out, q)


def test_offsets_beyond_32_bits():
    """Pages at the far end of a pool of over 4 GB a tensor."""
    page, heads, dim = 128, 4, 128
    lead = (1 << 32) // (page * heads * dim * 2) + 7
    b = Batch([2, 40], [300, 170], page, seed=2, lead_pages=lead)
    g = gen(12)
    w = b.whole()
    k, v = (torch.randn((w.tokens, heads, dim), generator=g, device="cuda").bfloat16() for _ in range(2))
    c = abi.KVCache.empty(b.num_pages, heads, page, dim)
    abi.dynrad_cache_write(c, k, v, *w.call())
    kr, vr = abi.dynrad_cache_read(c, *w.call(), w.tokens)
    assert torch.equal(kr, k) and torch.equal(vr, v)
    q = torch.randn((b.tokens, heads, dim), generator=g, device="cuda").bfloat16()
    o, lse = abi.dynrad_cache_attn(q, c, *b.call())
    torch.cuda.synchronize()
    check_device_status()
    kk, kv = ([f64(x)[w.cu_np[s]:w.cu_np[s + 1]] for s in range(2)] for x in (k, v))
    check_attention(o, lse, q, kk, kv, b, 1, 0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_video_written_and_attended_frame_by_frame(fmt):
    """The run a user makes: each frame's K and V are written, its tokens attend
    over all frames so far, pages taken as they are needed; at the end the history
    is read back and the block-sparse layer with every block kept gives the same
    as the cache's attention without a mask."""
    per, frames, heads, dim, page = 60, 5, 2, 64, 16
    n = per * frames
    b = Batch([n], [n], page, seed=4)
    g = gen(9)
    c = empty_cache(b, heads, dim, fmt)
    q, k, v = (torch.randn((n, heads, dim), generator=g, device="cuda").bfloat16() for _ in range(3))
    kept = []
    for x in (k, v):
        x = f64(x)
        kept.append(x if fmt == "bf16" else OC.stands_for(*OC.quantise(x, fmt), fmt))
    cu = torch.tensor([0, per], dtype=torch.int32, device="cuda")
    for f in range(frames):
        at = slice(f * per, (f + 1) * per)
        length = torch.tensor([(f + 1) * per], dtype=torch.int32, device="cuda")
        abi.dynrad_cache_write(c, k[at], v[at], b.table, cu, length)
        o, lse = abi.dynrad_cache_attn(q[at], c, b.table, cu, length, frame=per, window=3)
        step = object.__new__(Batch)
        step.ns, step.lens, step.cu_np = [per], [(f + 1) * per], np.array([0, per])
        check_attention(o, lse, q[at], [kept[0][:(f + 1) * per]], [kept[1][:(f + 1) * per]], step, per, 3)
    kr, vr = abi.dynrad_cache_read(c, *b.call(), n, head_major=True)
    assert np.array_equal(f64(kr.transpose(0, 1)), kept[0]) and np.array_equal(f64(vr.transpose(0, 1)), kept[1])
    o, lse = abi.dynrad_cache_attn(q, c, *b.call(), frame=0)
    rp, col = full_csr(-(-n // 64), heads)
    ob, lb = abi.dynrad_sparse_attn(q.transpose(0, 1).contiguous()[None], kr[None], vr[None], 64,
                                    torch.from_numpy(rp.astype(np.int32)).cuda(),
                                    torch.from_numpy(col.astype(np.int32)).cuda())
    torch.cuda.synchronize()
    check_device_status()
    # both within U_BF16 (sum softmax |v| + |o|) of the same value, |v| here at most 6
    assert (o.float() - ob[0].transpose(0, 1).float()).abs().max() <= 4 * 2.0 ** -8 * 6
    assert (lse - lb[0]).abs().max() <= 1e-3


def test_calls_on_other_streams_and_captured():
    b = Batch([1, 90, 3], [2700, 300, 64], 32, seed=7)
    g = gen(2)
    c, kk, kv = filled_cache(b, 2, 128, "fp8", g)
    q = torch.randn((b.tokens, 8, 128), generator=g, device="cuda").bfloat16()
    o_ref, lse_ref = abi.dynrad_cache_attn(q, c, *b.call())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o1, lse1 = abi.dynrad_cache_attn(q, c, *b.call())
    o2, lse2 = abi.dynrad_cache_attn(q, c, *b.call())       # at the same time, a workspace each
    torch.cuda.synchronize()
    for o, lse in ((o1, lse1), (o2, lse2)):
        assert torch.equal(o, o_ref) and torch.equal(lse, lse_ref)
    # the stream as an argument: what the call allocates is that stream's
    side.wait_stream(torch.cuda.current_stream())
    o3, lse3 = abi.dynrad_cache_attn(q, c, *b.call(), stream=side)
    k3, v3 = abi.dynrad_cache_read(c, *b.call(), b.tokens, stream=side)
    c3 = empty_cache(b, 2, 128, "fp8")
    side.wait_stream(torch.cuda.current_stream())
    abi.dynrad_cache_write(c3, k3, v3, *b.call(), stream=side)
    side.synchronize()
    assert torch.equal(o3, o_ref) and torch.equal(lse3, lse_ref)
    k4, _ = abi.dynrad_cache_read(c3, *b.call(), b.tokens)
    assert torch.equal(k4, k3)
    # a decode step captured once: write, attend; replayed with new inputs and lengths
    ns, lens = [1, 1, 1], [100, 40, 2700]
    b = Batch(ns, [n + 3 for n in lens], 32, seed=11, keys=1100)
    w = b.whole()
    k, v = (torch.randn((w.tokens, 2, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    c = empty_cache(b, 2, 128, "int8")
    abi.dynrad_cache_write(c, k, v, *w.call())
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nk, nv = (torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nq, out = (torch.zeros((3, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.zeros((8, 3), device="cuda")
    def step():
        abi.dynrad_cache_write(c, nk, nv, b.table, b.cu, length)
        abi.dynrad_cache_attn(nq, c, b.table, b.cu, length, out=out, lse=lse)
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kept = [OC.stands_for(*OC.quantise(f64(x), "int8"), "int8") for x in (k, v)]
    for r in range(3):
        length.copy_(torch.tensor([n + r + 1 for n in lens], dtype=torch.int32))
        for x in (nk, nv, nq):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        check_device_status()
        for x, y in zip(kept, (nk, nv)):
            for s in range(3):
                x[w.cu_np[s] + lens[s] + r] = OC.stands_for(*OC.quantise(f64(y[s]), "int8"), "int8")
        now = object.__new__(Batch)
        now.ns, now.lens, now.cu_np = ns, [n + r + 1 for n in lens], b.cu_np
        # position lens[s] - 1 was overwritten by the warm step's zeros
        for x in kept:
            for s in range(3):
                if r == 0:
                    x[w.cu_np[s] + lens[s] - 1] = 0.0
        check_attention(out, lse, nq, *([x[w.cu_np[s]:w.cu_np[s] + now.lens[s]] for s in range(3)] for x in kept),
                        now, 1, 0)


@pytest.mark.parametrize("ns,lens,group", [([1], [4000], 8), ([1, 2, 1], [3000, 1200, 15], 8), ([200, 1], [2500, 90], 3),
                                           ([40], [1100], 4)])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_one_workspace_for_calls_in_turn(ns, lens, group, fmt):
    """The caller's workspace: whatever it holds, and whichever call used it before."""
    b = Batch(ns, lens, 64, seed=3)
    g = gen(5)
    c, _, _ = filled_cache(b, 2, 128, fmt, g)
    q = torch.randn((b.tokens, 2 * group, 128), generator=g, device="cuda").bfloat16()
    need = abi.dynrad_cache_attn_workspace_bytes(c, len(ns), b.tokens, 2 * group)
    ws = torch.full((need // 4 + 64,), float("nan"), device="cuda")
    for frame in (1, 0):
        o_ref, lse_ref = abi.dynrad_cache_attn(q, c, *b.call(), frame=frame)
        for _ in range(2):
            o, lse = abi.dynrad_cache_attn(q, c, *b.call(), frame=frame, workspace=ws)
            assert torch.equal(o, o_ref) and torch.equal(lse, lse_ref)
    torch.cuda.synchronize()
    check_device_status()
    with pytest.raises(abi.DynradError):
        abi.dynrad_cache_attn(q, c, *b.call(), workspace=ws[:need // 4 - 1])
    with pytest.raises(abi.DynradError):
        abi.dynrad_cache_attn(q, c, *b.call(), workspace=ws[1:])
    with pytest.raises(ValueError):
        abi.dynrad_cache_attn(q, c, *b.call(), workspace=ws.cpu())
