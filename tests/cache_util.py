"""Batches over a paged K / V cache for the tests, and the oracle's answer with
its error bounds."""
from __future__ import annotations

import math

import numpy as np
import torch

from block_sparse_attention_candidate_b200 import abi
from oracle import cache as OC

DTYPE = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}
NOWHERE = (-1, 1 << 30, -(1 << 31), 0)   # entries of the table that must never be looked at


def f64(t):
    return t.detach().cpu().double().numpy()


class Batch:
    """Sequences of a call: n new tokens each, length with them, pages shuffled.
    Table entries behind a sequence's last page lead nowhere; `spare` columns
    and rows' padding are part of the table's stride."""

    def __init__(self, ns, lens, page, seed=0, tail=0, pad_cols=1, lead_pages=0, keys=0, skip=0):
        """keys: what the table's rows can hold at least (the library cuts items into
        parts where that is over 1024, chunks from 512 on); skip: rows before the first sequence's."""
        rng = np.random.default_rng(seed)
        self.ns, self.lens, self.page = list(ns), list(lens), page
        used = [-(-n // page) for n in lens]
        self.cols = max(used + [1, -(-keys // page)])
        self.num_pages = lead_pages + sum(used) + 2
        order = lead_pages + rng.permutation(self.num_pages - lead_pages)
        wide = np.array([[NOWHERE[(s + c) % 4] for c in range(self.cols + pad_cols)] for s in range(len(ns))],
                        dtype=np.int64).reshape(len(ns), self.cols + pad_cols)
        at = 0
        for s, u in enumerate(used):
            wide[s, :u] = order[at:at + u]
            at += u
        self.table_np = wide[:, :self.cols]
        self.cu_np = skip + np.concatenate([[0], np.cumsum(ns)]).astype(np.int64)
        self.tokens = int(self.cu_np[-1]) + tail
        self.tail = tail
        self.table = torch.from_numpy(wide.astype(np.int32)).cuda()[:, :self.cols]
        self.cu = torch.from_numpy(self.cu_np.astype(np.int32)).cuda()
        self.len = torch.tensor(list(lens), dtype=torch.int32, device="cuda")

    def call(self):
        return self.table, self.cu, self.len

    def whole(self):
        """The same cache seen as one call that has every position as a token."""
        b = object.__new__(Batch)
        b.__dict__.update(self.__dict__)
        b.ns = list(self.lens)
        b.cu_np = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int64)
        b.cu = torch.from_numpy(b.cu_np.astype(np.int32)).cuda()
        b.tokens, b.tail = int(b.cu_np[-1]), 0
        return b


def empty_cache(b, heads, dim, fmt, fill=True):
    """A cache whose every byte is a pattern that must not matter: NaN (bf16), or
    scale bytes of 255 (NaN) in the 8-bit formats."""
    c = abi.KVCache.empty(b.num_pages, heads, b.page, dim, DTYPE[fmt])
    if fill:
        for t in (c.k, c.v):
            t.view(torch.int16 if fmt == "bf16" else torch.uint8).fill_(-1 if fmt == "bf16" else 255)
        for t in (c.k_scale, c.v_scale):
            if t is not None:
                t.fill_(255)
    return c


def filled_cache(b, heads, dim, fmt, gen, scale=1.0, k=None, v=None):
    """A cache that holds seeded K, V at every position of the batch; also what it
    stands for: per sequence float64 [length, heads, dim] K and V."""
    w = b.whole()
    if k is None:
        k, v = ((scale * torch.randn((w.tokens, heads, dim), generator=gen, device="cuda")).bfloat16() for _ in range(2))
    c = empty_cache(b, heads, dim, fmt)
    abi.dynrad_cache_write(c, k, v, *w.call())
    kept = []
    for x in (k, v):
        x = f64(x)
        if fmt != "bf16":
            x = OC.stands_for(*OC.quantise(x, fmt), fmt)
        kept.append([x[w.cu_np[s]:w.cu_np[s + 1]] for s in range(len(b.ns))])
    return c, kept[0], kept[1]


U_BF16 = 2.0 ** -8     # half a step of bf16, relative
U_FP32 = 2.0 ** -24


def check_attention(o, lse, q, kept_k, kept_v, b, frame, window, scale=None):
    """o, lse of the batch's tokens against the oracle on what the cache holds.

    Bounds.  P is rounded to bf16 before it meets V (at most U_BF16 of it) and o
    once more, so |o - o*| <= U_BF16 (sum softmax |v| + |o*|), and a hundredth
    more for the second-order terms.  The logits are fp32 sums of D products
    (at most D + 4 roundings of sum |q k| scale), which shifts each softmax
    weight by at most twice that, relatively; exponentials and the two sums over
    n keys add (n + 16) fp32 half-steps at the worst, and P's and O's fp32
    arguments |logit| 2 log2(e) of them.  For lse the same without P."""
    d, heads = q.shape[2], q.shape[1]
    hk = kept_k[0].shape[1] if kept_k else 1
    g = heads // hk
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    qn, on, ln = f64(q), f64(o), f64(lse)
    for s in range(len(b.ns)):
        t0, t1 = int(b.cu_np[s]), int(b.cu_np[s + 1])
        for h in range(hk):
            rows = qn[t0:t1, h * g:(h + 1) * g]
            ref, lref, av, aqk = OC.attend(rows, kept_k[s][:, h], kept_v[s][:, h], b.lens[s], frame, window, scale)
            got, lgot = on[t0:t1, h * g:(h + 1) * g], ln[h * g:(h + 1) * g, t0:t1].T
            slack = U_FP32 * ((d + 8) * aqk + b.lens[s] + 16)
            tol = 1.01 * U_BF16 * (av + np.abs(ref)) + 2 * slack[..., None] * av + 1e-30
            assert np.array_equal(np.isnan(ref), np.isnan(got)), (s, h)
            ok = np.isfinite(ref)
            assert (np.abs(got - ref)[ok] <= tol[ok]).all(), (s, h, np.abs(got - ref)[ok].max())
            none = lref == -math.inf
            assert np.array_equal(none, lgot == -math.inf), (s, h)
            assert (got[none] == 0).all()
            assert np.array_equal(np.isnan(lref), np.isnan(lgot))
            live = np.isfinite(lref)
            ltol = 2 * slack + 4 * U_FP32 * np.abs(np.where(live, lref, 0.0))
            assert (np.abs(lgot[live] - lref[live]) <= ltol[live]).all(), (s, h, np.abs(lgot[live] - lref[live]).max())
