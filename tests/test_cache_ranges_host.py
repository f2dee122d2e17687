"""Numbers past 32 bits at the binding of the cache calls: refused, never taken modulo 2^32."""
import pytest
import torch

from block_sparse_attention_candidate_b200 import abi

WRAPS = [2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 40 + 3]


def _call():
    kv = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    i32 = torch.int32
    seqs = torch.zeros((3, 4), dtype=i32), torch.zeros(4, dtype=i32), torch.zeros(3, dtype=i32)
    return abi.KVCache(kv, kv.clone()), torch.zeros((9, 4, 64), dtype=torch.bfloat16), seqs


@pytest.mark.parametrize("n", WRAPS + [-2 ** 31 - 5, -2 ** 32])
def test_frame_and_window(n):
    cache, q, seqs = _call()
    with pytest.raises(ValueError, match="frame and window"):
        abi.dynrad_cache_attn(q, cache, *seqs, frame=n)
    with pytest.raises(ValueError, match="frame and window"):
        abi.dynrad_cache_attn(q, cache, *seqs, frame=1, window=n)


@pytest.mark.parametrize("n", WRAPS)
def test_tokens_sequences_and_pages(n):
    cache, q, (table, cu, length) = _call()
    with pytest.raises(ValueError, match="2\\^31"):
        abi._cache_seqs(cache, table, cu, length, n)
    k = q[:1, :2].expand(n, 2, 64)
    with pytest.raises(ValueError, match="2\\^31"):
        abi.dynrad_cache_write(cache, k, k, table, cu, length)
    with pytest.raises(ValueError, match="2\\^31"):
        abi._cache_seqs(cache, table[:, :1].expand(3, n), cu, length, 9)


@pytest.mark.parametrize("n", WRAPS + [-1])
def test_workspace_of_a_call_that_can_not_be_made(n):
    cache, _, _ = _call()
    assert abi.dynrad_cache_attn_workspace_bytes(cache, 3, 9, 4) > 0
    assert abi.dynrad_cache_attn_workspace_bytes(cache, n, 9, 4) == 0
    assert abi.dynrad_cache_attn_workspace_bytes(cache, 3, n, 4) == 0
    assert abi.dynrad_cache_attn_workspace_bytes(cache, 3, 9, 2 * n) == 0
