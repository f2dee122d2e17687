"""Cache attention where a seen NaN or infinity meets logits far above it: what
a row sees reaches it however its keys are shared out (over the warps of a CTA, the
two accumulators of an item with rows for one tile, the parts of a cut item)."""
import math

import pytest
import torch

from block_sparse_attention_candidate_b200 import abi
from cache_util import Batch, check_attention, filled_cache
from gpu_util import check_device_status
from oracle import cache as OC

pytestmark = pytest.mark.gpu

# (new tokens, lengths, query heads, K / V heads): single tokens in one and in two column
# tiles, an item with rows for one tile, an item of two; short and long
CALLS = {
    "token": ([1, 1], [900, 700], 4, 2),
    "token16": ([2, 2], [900, 640], 8, 1),
    "narrow": ([40], [450], 2, 2),
    "wide": ([300], [450], 2, 2),
    "long token": ([1, 1], [3000, 2100], 4, 2),
    "long token16": ([2, 2], [3000, 2100], 8, 1),
    "long narrow": ([40], [3000], 2, 2),
    "long wide": ([300], [3000], 2, 2),
}
# (position of what is not finite, position of the strong key): in neighbouring blocks of
# keys and steps, and far apart, either way round; negative: from the sequence's end
PLACES = [(5, 40), (5, 150), (150, 5), (20, 600), (600, 20), (3, -60), (-60, 3), (-2, 100)]


def strong_case(ns, lens, heads, kv_heads, dim, fmt, bad_at, strong_at):
    """q of 4s; keys whose logits are of order 1, but for one of 16 sqrt(dim) (128 or
    more: a weight of 1 there is under 2^-126 for every other key)."""
    b = Batch(ns, lens, 32, seed=2)
    g = torch.Generator("cuda").manual_seed(dim + len(ns))
    w = b.whole()
    k = (0.25 * torch.randn((w.tokens, kv_heads, dim), generator=g, device="cuda")).bfloat16()
    v = torch.randn((w.tokens, kv_heads, dim), generator=g, device="cuda").bfloat16()
    q = torch.full((b.tokens, heads, dim), 4.0, dtype=torch.bfloat16, device="cuda")
    bad = []
    for s, length in enumerate(lens):
        bad.append(bad_at % length)
        k[int(w.cu_np[s]) + strong_at % length] = 4.0
    return b, g, k, v, q, bad, [int(w.cu_np[s]) + x for s, x in enumerate(bad)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("bad_at,strong_at", PLACES)
def test_what_a_row_sees_reaches_it_under_any_weight(fmt, dim, call, bad_at, strong_at):
    ns, lens, heads, kv_heads = CALLS[call]
    b, g, k, v, q, bad, rows = strong_case(ns, lens, heads, kv_heads, dim, fmt, bad_at, strong_at)
    for what in ("k", "v"):
        k2, v2 = k.clone(), v.clone()
        (k2 if what == "k" else v2)[rows, :, 5] = math.nan
        c, kk, kv = filled_cache(b, kv_heads, dim, fmt, g, k=k2, v=v2)
        o, lse = abi.dynrad_cache_attn(q, c, *b.call())
        torch.cuda.synchronize()
        check_device_status()
        check_attention(o, lse, q, kk, kv, b, 1, 0)      # NaN in the same places, the rest within bounds


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("bad_at,strong_at", PLACES)
def test_a_seen_infinity_is_not_lost(call, bad_at, strong_at):
    """An infinity in V under a weight that fp32 holds as 0: infinity or NaN, never finite."""
    ns, lens, heads, kv_heads = CALLS[call]
    b, g, k, v, q, bad, rows = strong_case(ns, lens, heads, kv_heads, 64, "bf16", bad_at, strong_at)
    clean, kk, kv = filled_cache(b, kv_heads, 64, "bf16", g, k=k, v=v)
    o_ref, lse_ref = abi.dynrad_cache_attn(q, clean, *b.call())
    v[rows, :, 5] = math.inf
    c, _, _ = filled_cache(b, kv_heads, 64, "bf16", g, k=k, v=v)
    o, lse = abi.dynrad_cache_attn(q, c, *b.call())
    torch.cuda.synchronize()
    check_device_status()
    assert torch.equal(lse, lse_ref)
    for s in range(len(ns)):
        for i in range(ns[s]):
            lo, hi = OC.seen(1, 0, lens[s] - ns[s] + i, lens[s])
            t = int(b.cu_np[s]) + i
            if lo <= bad[s] < hi:
                assert not torch.isfinite(o[t, :, 5]).any(), (s, i)
                assert torch.equal(o[t, :, 6:], o_ref[t, :, 6:])
            else:
                assert torch.equal(o[t], o_ref[t]), (s, i)
