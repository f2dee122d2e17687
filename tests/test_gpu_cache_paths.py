"""Paged K / V cache on the GPU: the kernels' less usual paths, against the float64
oracle (bounds of cache_util.check_attention; stored and read bytes exactly)."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_candidate_b200 import abi
from cache_util import Batch, check_attention, empty_cache, f64, filled_cache
from gpu_util import check_device_status
from oracle import cache as OC
from test_gpu_cache import laid_out, odd_values

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "fp8", "int8"]


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def positions(b):
    """(rows, page, slot) of the tokens that have a position, and the rows that have none."""
    rows, pages, slots, none = [], [], [], []
    for s, (n, length) in enumerate(zip(b.ns, b.lens)):
        at = np.arange(length - n, length)
        row = int(b.cu_np[s]) + np.arange(n)
        none.append(row[at < 0])
        row, at = row[at >= 0], at[at >= 0]
        rows.append(row)
        pages.append(b.table_np[s, at // b.page])
        slots.append(at % b.page)
    return (np.concatenate(x) for x in (rows, pages, slots, none))


# more tokens than the SMs have room for CTAs, so that a CTA takes several; the last takes fewer
MANY = {
    "601": ([600, 1], [650, 1]),
    "1187": ([700, 0, 9, 478], [690, 5, 100, 478]),
    "4803": ([1, 4000, 30, 772], [200, 4000, 12, 801]),
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,heads", [(64, 1), (64, 3), (128, 2), (128, 9)])
@pytest.mark.parametrize("name", list(MANY))
@pytest.mark.parametrize("page,layout", [(16, "thd"), (128, "htd"), (64, "wide")])
def test_write_and_read_of_many_tokens(fmt, dim, heads, name, page, layout):
    ns, lens = MANY[name]
    b = Batch(ns, lens, page, seed=3, tail=5, skip=2)
    x = [odd_values((b.tokens, heads, dim), 70 + i).cuda() for i in range(2)]
    c = empty_cache(b, heads, dim, fmt)
    abi.dynrad_cache_write(c, *(laid_out(y, layout) for y in x), *b.call())
    rows, pages, slots, none = positions(b)
    raw = torch.int16 if fmt == "bf16" else torch.uint8
    back = []
    for y, held, scale in zip(x, (c.k, c.v), (c.k_scale, c.v_scale)):
        want = np.full(held.shape, -1 if fmt == "bf16" else 255, dtype=np.int16 if fmt == "bf16" else np.uint8)
        if fmt == "bf16":
            want[pages, :, slots] = y.view(torch.int16).cpu().numpy()[rows]
            back.append(f64(y))
        else:
            code, byte = OC.quantise(f64(y), fmt)
            want[pages, :, slots] = code[rows]
            wscale = np.full(scale.shape, 255, dtype=np.uint8)
            wscale[pages, :, slots] = byte[rows]
            assert np.array_equal(scale.cpu().numpy(), wscale)
            back.append(OC.stands_for(code, byte, fmt))
        assert np.array_equal(held.view(raw).cpu().numpy(), want)
    out = [laid_out(torch.full((b.tokens, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda"), layout)
           for _ in range(2)]
    abi.dynrad_cache_read(c, *b.call(), out=tuple(out))
    torch.cuda.synchronize()
    check_device_status()
    for o, kept in zip(out, back):
        want = np.full((b.tokens, heads, dim), 7.0)      # rows before, behind and between: nobody's
        want[rows], want[none] = kept[rows], 0.0
        assert np.array_equal(f64(o), want, equal_nan=True)


# (new tokens, lengths, query heads, K / V heads): 9 to 16 rows of a sequence and K / V head
SIXTEEN = [([1, 1, 1], [900, 33, 1], 9, 1), ([1, 1], [520, 40], 24, 2), ([1, 1], [260, 700], 16, 1),
           ([2, 2, 1], [640, 77, 3], 16, 2), ([2, 2], [1, 300], 8, 1), ([16, 15, 3], [800, 15, 100], 2, 2),
           ([5, 4], [333, 450], 3, 1)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("which", range(len(SIXTEEN)))
@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("frame,window", [(1, 0), (7, 30)])
def test_nine_to_sixteen_rows(fmt, dim, which, long, frame, window):
    ns, lens, heads, kv_heads = SIXTEEN[which]
    if long:     # items are cut into parts
        lens = [n + 1400 * (i + 1) for i, n in enumerate(lens)]
    b = Batch(ns, lens, 32, seed=which, tail=1)
    g = gen(which)
    c, kk, kv = filled_cache(b, kv_heads, dim, fmt, g)
    q = torch.randn((b.tokens, heads, dim), generator=g, device="cuda").bfloat16()
    need = abi.dynrad_cache_attn_workspace_bytes(c, len(ns), b.tokens, heads)
    ws = torch.full((need // 4,), math.nan, device="cuda")
    o, lse = abi.dynrad_cache_attn(q, c, *b.call(), frame=frame, window=window, workspace=ws)
    torch.cuda.synchronize()
    check_device_status()
    check_attention(o, lse, q, kk, kv, b, frame, window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ns,lens,heads,kv_heads,dim,frame,window", [
    ([1] * 40 + [300], [1 + 13 * i for i in range(40)] + [700], 2, 2, 128, 1, 0),
    ([1] * 60 + [200, 0, 3], [300 - i for i in range(60)] + [1500, 9, 2], 8, 2, 64, 1, 0),
    ([1] * 30 + [170], [64] * 30 + [1200], 1, 1, 64, 50, 6),
])
def test_a_chunk_among_many_single_tokens(fmt, ns, lens, heads, kv_heads, dim, frame, window):
    """The average sends the chunk through the single tokens' kernel."""
    b = Batch(ns, lens, 16, seed=2, tail=3)
    g = gen(len(ns))
    c, kk, kv = filled_cache(b, kv_heads, dim, fmt, g)
    q = torch.randn((b.tokens, heads, dim), generator=g, device="cuda").bfloat16()
    o, lse = abi.dynrad_cache_attn(q, c, *b.call(), frame=frame, window=window)
    torch.cuda.synchronize()
    check_device_status()
    check_attention(o, lse, q, kk, kv, b, frame, window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seqs,heads,kv_heads,dim", [(150, 64, 8, 64), (80, 40, 8, 64), (100, 96, 12, 128)])
def test_large_ragged_batches_of_wide_groups(fmt, seqs, heads, kv_heads, dim):
    """5 to 8 query heads to a K / V head: an item a token, uncut; one sequence far longer."""
    lens = [1 + (37 * i) % 150 for i in range(seqs)]
    lens[seqs // 2] = 2500
    b = Batch([1] * seqs, lens, 16, seed=4)
    g = gen(seqs)
    c, kk, kv = filled_cache(b, kv_heads, dim, fmt, g)
    q = torch.randn((b.tokens, heads, dim), generator=g, device="cuda").bfloat16()
    o, lse = abi.dynrad_cache_attn(q, c, *b.call())
    torch.cuda.synchronize()
    check_device_status()
    check_attention(o, lse, q, kk, kv, b, 1, 0)


@pytest.mark.parametrize("fmt,k_exp,v_exp", [("fp8", (0, 60), (-20, 8, 90)), ("fp8", (9, 100), (60,)),
                                             ("int8", (0, 124), (-60, 0, 80)), ("int8", (124, 124), (100,)),
                                             ("int8", (0, 126), (-60, 0, 80)), ("int8", (126, 126), (100,))])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("ns,lens,heads,kv_heads", [([1, 1], [700, 90], 4, 1), ([2, 2], [1800, 90], 8, 1),
                                                    ([70], [300], 2, 2), ([300, 9], [800, 400], 2, 2)])
def test_large_scales_in_attention(fmt, k_exp, v_exp, dim, ns, lens, heads, kv_heads):
    """Scales whose factor takes two steps (2^8 and over in e4m3, 2^121 in int8), beside
    small ones: the halves of K's channels at 2^k_exp, V's tokens in turn at 2^v_exp; q's
    channels make up for K's, so that logits are of order 1.  int8 at 2^124 stays just below
    such scales; at 2^126 q and the logit scale share the making up, since q's numbers would
    be subnormal."""
    b = Batch(ns, lens, 32, seed=6)
    g = gen(dim + len(k_exp))
    w = b.whole()
    half = torch.arange(dim, device="cuda") >= dim // 2
    ke = torch.where(half, float(k_exp[1]), float(k_exp[0]))
    ve = torch.tensor(v_exp, device="cuda", dtype=torch.float32)[torch.arange(w.tokens, device="cuda") % len(v_exp)]
    k = torch.randn((w.tokens, kv_heads, dim), generator=g, device="cuda")
    lift = 6 if k_exp[1] == 126 else 0
    k = torch.ldexp(k.clamp(-3, 3) if lift else k, ke).bfloat16()
    v = torch.ldexp(torch.randn((w.tokens, kv_heads, dim), generator=g, device="cuda"), ve[:, None, None]).bfloat16()
    q = torch.ldexp(torch.randn((b.tokens, heads, dim), generator=g, device="cuda").clamp(-3, 3), lift - ke).bfloat16()
    scale = 2.0 ** -lift / math.sqrt(dim)
    c, kk, kv = filled_cache(b, kv_heads, dim, fmt, g, k=k, v=v)
    odd = 134 if fmt == "fp8" else 247
    assert bool(((c.k_scale > odd) & (c.k_scale != 255)).any()) == (124 not in k_exp)
    o, lse = abi.dynrad_cache_attn(q, c, *b.call(), scale=scale)
    torch.cuda.synchronize()
    check_device_status()
    check_attention(o, lse, q, kk, kv, b, 1, 0, scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("ns,lens", [([2, 3], [112, 33]), ([2, 3], [2300, 1500]), ([100, 1], [150, 140]),
                                     ([300], [420]), ([300], [2600])])
@pytest.mark.parametrize("frame,window", [(1, 0), (1, 20), (16, 2)])
def test_values_that_some_rows_see(fmt, dim, ns, lens, frame, window):
    """NaN in V at the last positions and further back: rows that see it are NaN there."""
    b = Batch(ns, lens, 32, seed=8)
    g = gen(dim)
    w = b.whole()
    k, v = (torch.randn((w.tokens, 2, dim), generator=g, device="cuda").bfloat16() for _ in range(2))
    for s, length in enumerate(lens):
        at = int(w.cu_np[s])
        v[at + length - 1, :, 3] = math.nan
        v[at + max(length - 17, 0), 0, dim - 1] = math.nan
        v[at + max(length - ns[s], 0), 1, 33] = math.nan
    q = torch.randn((b.tokens, 6, dim), generator=g, device="cuda").bfloat16()
    c, kk, kv = filled_cache(b, 2, dim, fmt, g, k=k, v=v)
    o, lse = abi.dynrad_cache_attn(q, c, *b.call(), frame=frame, window=window)
    torch.cuda.synchronize()
    check_device_status()
    for x in kv:     # the oracle's 0 * NaN of rows that do not see it does not arise: it cuts K and V first
        assert np.isnan(x).any()
    check_attention(o, lse, q, kk, kv, b, frame, window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ns", [[1, 1, 1], [40, 3, 130]])
def test_sequences_that_share_pages(fmt, ns):
    """A common beginning: the same pages in three rows of the table."""
    page, dim, shared = 32, 128, 160
    lens = [shared + n + 5 * i for i, n in enumerate(ns)]
    b = Batch(ns, lens, page, seed=1)
    g = gen(11)
    w = b.whole()
    k, v = (torch.randn((w.tokens, 2, dim), generator=g, device="cuda").bfloat16() for _ in range(2))
    for x in (k, v):
        for s in (1, 2):
            x[int(w.cu_np[s]):int(w.cu_np[s]) + shared] = x[:shared]
    c, kk, kv = filled_cache(b, 2, dim, fmt, g, k=k, v=v)
    table = b.table.clone()
    table[1:, :shared // page] = table[:1, :shared // page]
    q = torch.randn((b.tokens, 4, dim), generator=g, device="cuda").bfloat16()
    o, lse = abi.dynrad_cache_attn(q, c, table, b.cu, b.len)
    torch.cuda.synchronize()
    check_device_status()
    check_attention(o, lse, q, kk, kv, b, 1, 0)
