"""Paged K / V cache without a GPU: the calls' refusals, the workspace size, the
struct layouts, and the oracle's own pins."""
import ctypes
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_candidate_b200 import abi
from oracle import cache as OC
from test_abi_host import _c_layout

P = 0x10000


def _cache(**kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, num_pages=10, heads=2, page=64, dim=128, format=1)
    a.update(kw)
    return abi.DynradKvCache(*a.values())


def _seqs(**kw):
    a = dict(page_table=P, cu_seq=P, kv_len=P, table_stride=4, num_seqs=3, max_pages=4, num_tokens=7)
    a.update(kw)
    return abi.DynradSeqs(*a.values())


BAD_STRUCTS = [
    (dict(k=None), {}, 1), (dict(v=None), {}, 1), (dict(k=P + 8), {}, 1), (dict(k_scale=None), {}, 1),
    (dict(v_scale=P + 4), {}, 1), (dict(format=3), {}, 1), (dict(format=-1), {}, 1), (dict(num_pages=0), {}, 1),
    (dict(heads=0), {}, 1), (dict(dim=96), {}, 2), (dict(dim=256), {}, 2), (dict(page=48), {}, 2),
    (dict(page=8), {}, 2), (dict(page=256), {}, 2), (dict(heads=1 << 16), {}, 2), (dict(num_pages=1 << 25), {}, 2),
    ({}, dict(cu_seq=None), 1), ({}, dict(page_table=None), 1), ({}, dict(kv_len=None), 1),
    ({}, dict(num_seqs=-1), 1), ({}, dict(num_tokens=-1), 1), ({}, dict(max_pages=-1), 1),
    ({}, dict(table_stride=3), 1), ({}, dict(max_pages=1 << 26, table_stride=1 << 26), 2),
]


@pytest.mark.parametrize("ckw,skw,want", BAD_STRUCTS)
def test_bad_cache_or_sequences_refused_before_launch(ckw, skw, want):
    L, c, s = abi.lib(), _cache(**ckw), _seqs(**skw)
    c, s = ctypes.byref(c), ctypes.byref(s)
    assert L.dynrad_cache_write(c, s, P, 256, 128, P, 256, 128, None) == want
    assert L.dynrad_cache_read(c, s, P, 256, 128, P, 256, 128, None) == want
    assert L.dynrad_cache_attn(c, s, P, 512, 128, 4, 1, 0, 0.0, P, 512, 128, P, P, 1 << 40, None) == want
    assert L.dynrad_cache_write(None, s, P, 256, 128, P, 256, 128, None) == 1
    assert L.dynrad_cache_write(c, None, P, 256, 128, P, 256, 128, None) == 1


def test_bad_operands_refused_before_launch():
    L, c, s = abi.lib(), ctypes.byref(_cache()), ctypes.byref(_seqs())
    for f in (L.dynrad_cache_write, L.dynrad_cache_read):
        assert f(c, s, None, 256, 128, P, 256, 128, None) == 1
        assert f(c, s, P, 256, 128, None, 256, 128, None) == 1
        assert f(c, s, P + 2, 256, 128, P, 256, 128, None) == 1
        assert f(c, s, P, 250, 128, P, 256, 128, None) == 1
        assert f(c, s, P, 256, 128, P, 256, 124, None) == 1
        assert f(c, s, P, -256, 128, P, 256, 128, None) == 1

    def attn(q=P, qt=512, qh=128, heads=4, frame=1, window=0, scale=0.0, o=P, ot=512, oh=128, lse=P, ws=P,
             ws_bytes=1 << 40):
        return L.dynrad_cache_attn(c, s, q, qt, qh, heads, frame, window, scale, o, ot, oh, lse, ws, ws_bytes, None)

    assert attn(q=None) == 1 and attn(o=None) == 1 and attn(lse=None) == 1 and attn(ws=None) == 1
    assert attn(q=P + 8) == 1 and attn(o=P + 2) == 1 and attn(ws=P + 16) == 1
    assert attn(heads=3) == 1 and attn(heads=0) == 1
    assert attn(heads=258) == 2                                  # 129 query heads to a K / V head
    assert attn(frame=-1) == 1 and attn(window=-1) == 1 and attn(frame=0, window=2) == 1
    assert attn(scale=-1.0) == 1 and attn(scale=math.nan) == 1 and attn(scale=math.inf) == 1
    assert attn(scale=1e-40) == 1 and attn(scale=3e38) == 1
    assert attn(qt=500) == 1 and attn(oh=4) == 1 and attn(qt=0) == 1 and attn(qh=0) == 1
    assert attn(ws_bytes=16) == abi.DYNRAD_ERR_CAPACITY
    assert L.dynrad_cache_attn_workspace_bytes(c, 3, 7, 3) == 0
    assert L.dynrad_cache_attn_workspace_bytes(c, -1, 7, 4) == 0
    assert L.dynrad_cache_attn_workspace_bytes(None, 3, 7, 4) == 0
    assert L.dynrad_cache_attn_workspace_bytes(c, 3, 7, 4) > 0


def test_calls_without_tokens_or_sequences_do_nothing():
    L, c = abi.lib(), ctypes.byref(_cache())
    for s in (_seqs(num_tokens=0), _seqs(num_seqs=0, page_table=None, cu_seq=None, kv_len=None)):
        s = ctypes.byref(s)
        assert L.dynrad_cache_write(c, s, None, 0, 0, None, 0, 0, None) == 0
        assert L.dynrad_cache_read(c, s, None, 0, 0, None, 0, 0, None) == 0
        assert L.dynrad_cache_attn(c, s, None, 0, 0, 4, 1, 0, 0.0, None, 0, 0, None, None, 0, None) == 0


@pytest.mark.parametrize("struct,cls", [("dynrad_kv_cache", abi.DynradKvCache), ("dynrad_seqs", abi.DynradSeqs)])
def test_struct_layouts_match_c(struct, cls):
    names = [f[0] for f in cls._fields_]
    got = _c_layout(struct, names)
    assert got[0] == ctypes.sizeof(cls)
    for n, off in zip(names, got[1:]):
        assert getattr(cls, n).offset == off, n


def test_binding_checks_tensors():
    def t(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype)

    kv = t(5, 2, 16, 64)
    cache = abi.KVCache(kv, kv.clone())
    q8 = t(5, 2, 16, 64, dtype=torch.int8)
    sc = t(5, 2, 16, 2, dtype=torch.uint8)
    abi.KVCache(q8, q8.clone(), sc, sc.clone())
    i32 = torch.int32
    table, cu, ln = t(3, 4, dtype=i32), t(4, dtype=i32), t(3, dtype=i32)
    abi._cache_seqs(cache, table, cu, ln, 9)
    assert abi._cache_seqs(cache, t(3, 9, dtype=i32)[:, :4], cu, ln, 9).table_stride == 9
    assert abi._cache_rows(cache, "k", t(9, 2, 64), 2) == (128, 64)
    assert abi._cache_rows(cache, "k", t(2, 9, 64).transpose(0, 1), 2) == (64, 576)
    assert abi._cache_rows(cache, "k", t(9, 1, 64).expand(9, 2, 64), 2) == (64, 0)
    bad = [
        lambda: abi.KVCache(kv, t(5, 2, 16, 128)),
        lambda: abi.KVCache(kv.float(), kv.float()),
        lambda: abi.KVCache(kv.transpose(1, 2), kv.transpose(1, 2)),
        lambda: abi.KVCache(q8, q8),
        lambda: abi.KVCache(q8, q8, sc, sc[..., :1]),
        lambda: abi.KVCache(kv, kv, sc, sc),
        lambda: abi._cache_seqs(cache, table.long(), cu, ln, 9),
        lambda: abi._cache_seqs(cache, table, cu[:3], ln, 9),
        lambda: abi._cache_seqs(cache, table, cu, t(4, dtype=i32), 9),
        lambda: abi._cache_seqs(cache, table.t().contiguous().t(), cu, ln, 9),
        lambda: abi._cache_seqs(cache, table, t(8, dtype=i32)[::2], ln, 9),
        lambda: abi._cache_rows(cache, "k", t(9, 3, 64), 2),
        lambda: abi._cache_rows(cache, "k", t(9, 2, 128), 2),
        lambda: abi._cache_rows(cache, "k", t(9, 2, 64).float(), 2),
        lambda: abi._cache_rows(cache, "k", t(9, 2, 128)[..., ::2], 2),
        lambda: abi._cache_rows(cache, "k", t(9, 2, 68)[..., :64], 2),
        lambda: abi._cache_rows(cache, "v", t(8, 2, 64), 2, 9),
        lambda: abi._cache_rows(cache, "out", t(9, 1, 64).expand(9, 2, 64), 2, written=True),
        lambda: abi.dynrad_cache_write(cache, t(9, 2, 64), t(9, 2, 64), table, cu, ln),     # not on a CUDA device
        lambda: abi.dynrad_cache_read(cache, table, cu, ln),
        lambda: abi.dynrad_cache_read(cache, table, cu, ln, 8, out=(t(9, 2, 64), t(9, 2, 64))),
        lambda: abi.dynrad_cache_attn(t(9, 3, 64), cache, table, cu, ln),
        lambda: abi.dynrad_cache_attn(t(9, 1, 64).expand(9, 4, 64), cache, table, cu, ln),
        lambda: abi.dynrad_cache_attn(t(9, 4, 64), cache, table, cu, ln, lse=t(4, 8, dtype=torch.float32)),
        lambda: abi.dynrad_cache_attn(t(9, 4, 64), cache, table, cu, ln, lse=t(4, 9)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)


def test_binding_checks_the_workspace():
    i32 = torch.int32
    kv = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    cache = abi.KVCache(kv, kv.clone())
    q = torch.zeros((9, 4, 64), dtype=torch.bfloat16)
    seqs = torch.zeros((3, 4), dtype=i32), torch.zeros(4, dtype=i32), torch.zeros(3, dtype=i32)
    need = abi.dynrad_cache_attn_workspace_bytes(cache, 3, 9, 4)
    assert need > 0 and abi.dynrad_cache_attn_workspace_bytes(cache, 3, 9, 3) == 0
    with pytest.raises(ValueError, match="workspace"):
        abi.dynrad_cache_attn(q, cache, *seqs, workspace=torch.zeros(2 * need, dtype=torch.uint8)[::2])


# ------------------------------------------------------------------ the oracle's pins --
def test_oracle_e4m3_is_torchs():
    y = torch.cat([torch.linspace(-448, 448, 40001), torch.logspace(-12, 8.8, 20001, base=2),
                   -torch.logspace(-12, 8.8, 20001, base=2), torch.tensor([0.0, -0.0])]).clamp(-448, 448)
    want = y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OC.round_e4m3(y.double().numpy()), want)
    codes = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    vals = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    one = np.full((codes.size, 1), 127, dtype=np.uint8)
    wide = np.repeat(codes[:, None], 32, 1)
    assert np.array_equal(OC.stands_for(wide, one, "fp8")[:, 0], vals)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
def test_oracle_quantisation_bounds(fmt):
    """Least scale within range, every channel off by at most half a step, exact in bf16."""
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((300, 64)) * np.exp2(rng.integers(-100, 100, (300, 1)))).bfloat16()
    x = x.double().numpy()
    code, byte = OC.quantise(x, fmt)
    s = np.exp2(byte.astype(np.float64) - 127)
    a = np.abs(x.reshape(300, 2, 32)).max(-1)
    assert (a <= OC.LIMIT[fmt] * s).all() and (a > OC.LIMIT[fmt] * s / 2).all()
    back = OC.stands_for(code, byte, fmt)
    step = np.repeat(s, 32, -1) * (1.0 if fmt == "int8" else np.exp2(np.floor(np.log2(np.maximum(
        np.abs(x) / np.repeat(s, 32, -1), 2.0 ** -6))) - 3))
    assert (np.abs(back - x) <= step / 2).all()
    assert np.array_equal(torch.from_numpy(back).bfloat16().double().numpy(), back)


def test_oracle_attention_is_a_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 2, 8)), rng.standard_normal((9, 8)), rng.standard_normal((9, 8))
    o, lse, _, _ = OC.attend(q, k, v, 9, 1, 0, 0.5)
    for i in range(4):
        for h in range(2):
            a = k[:6 + i] @ q[i, h] * 0.5
            assert np.allclose(lse[i, h], np.log(np.exp(a).sum()))
            assert np.allclose(o[i, h], torch.softmax(torch.from_numpy(a), 0).numpy() @ v[:6 + i])
    assert OC.seen(4, 0, 5, 100) == (0, 8) and OC.seen(4, 2, 9, 10) == (4, 10) and OC.seen(1, 0, -1, 5) == (0, 0)
    assert OC.seen(0, 0, -3, 5) == (0, 5)
