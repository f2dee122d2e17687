"""Outputs of the cache calls beside their inputs in memory: overlapping tensors are
refused, slices of one tensor give what separate tensors give."""
import pytest
import torch

from block_sparse_attention_candidate_b200 import abi
from cache_util import Batch, filled_cache
from gpu_util import check_device_status

pytestmark = pytest.mark.gpu


def test_out_beside_q_in_one_tensor():
    b = Batch([3, 70], [90, 300], 32, seed=5)
    g = torch.Generator("cuda").manual_seed(3)
    c, _, _ = filled_cache(b, 2, 64, "bf16", g)
    T, H, D = b.tokens, 4, 64
    q = torch.randn((T, H, D), generator=g, device="cuda").bfloat16()
    o_ref, lse_ref = abi.dynrad_cache_attn(q, c, *b.call())
    for shape, cut in (((T, 2 * H, D), lambda x, i: x[:, i * H:(i + 1) * H]),
                       ((T, 2, H, D), lambda x, i: x[:, i]),
                       ((2 * H, T, D), lambda x, i: x[i::2].transpose(0, 1)),
                       ((2, T, H, D), lambda x, i: x[i])):
        both = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
        cut(both, 0).copy_(q)
        o, lse = abi.dynrad_cache_attn(cut(both, 0), c, *b.call(), out=cut(both, 1))
        assert torch.equal(o, o_ref) and torch.equal(lse, lse_ref) and torch.equal(cut(both, 0), q)
    wide = torch.zeros((T + 1, H, D), dtype=torch.bfloat16, device="cuda")
    for inp, out in ((wide[:-1], wide[:-1]), (wide[:-1], wide[1:]), (wide[1:], wide[:-1])):
        with pytest.raises(abi.DynradError):
            abi.dynrad_cache_attn(inp, c, *b.call(), out=out)
    torch.cuda.synchronize()
    check_device_status()


def test_read_into_slices_of_one_tensor():
    b = Batch([3, 70], [90, 300], 32, seed=5)
    g = torch.Generator("cuda").manual_seed(4)
    c, _, _ = filled_cache(b, 2, 64, "int8", g)
    k, v = abi.dynrad_cache_read(c, *b.call(), b.tokens)
    both = torch.zeros((b.tokens, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    abi.dynrad_cache_read(c, *b.call(), out=(both[:, 0], both[:, 1]))
    assert torch.equal(both[:, 0], k) and torch.equal(both[:, 1], v)
    with pytest.raises(abi.DynradError):
        abi.dynrad_cache_read(c, *b.call(), out=(k, k))
    torch.cuda.synchronize()
    check_device_status()
