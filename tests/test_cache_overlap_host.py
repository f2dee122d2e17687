"""Outputs of the cache calls that overlap an input, another output or themselves are
refused before any launch (csrc/rows.h, checked against every pair of rows with the host
C++ compiler)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from block_sparse_attention_candidate_b200 import abi
from test_cache_host import P, _cache, _seqs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "native", "rows_test.cpp")
INC = os.path.join(ROOT, "block_sparse_attention_candidate_b200", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_rows_against_every_pair(tmp_path):
    exe = str(tmp_path / "rows_test")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", INC, SRC, "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


# 7 tokens of 4 heads of 128 channels: 7168 bytes
Q, SIZE = 1 << 30, 7168


def _attn(q, qs, o, os_):
    c, s = _cache(heads=2), _seqs(num_tokens=7)
    return abi.lib().dynrad_cache_attn(ctypes.byref(c), ctypes.byref(s), q, *qs, 4, 1, 0, 0.0, o, *os_, P, P, 1 << 40,
                                       None)


def _read(k, ks, v, vs):
    c, s = _cache(heads=4), _seqs(num_tokens=7)
    return abi.lib().dynrad_cache_read(ctypes.byref(c), ctypes.byref(s), k, *ks, v, *vs, None)


@pytest.mark.parametrize("call", [_attn, _read])
@pytest.mark.parametrize("a,b", [((512, 128), (512, 128)), ((512, 128), (128, 896)), ((128, 896), (512, 128))])
def test_operands_that_overlap_are_refused(call, a, b):
    for at in (Q, Q + 16, Q + SIZE - 16, Q - SIZE + 16):
        assert call(Q, a, at, b) == abi.DYNRAD_ERR_INVALID_ARG


@pytest.mark.parametrize("strides", [(0, 128), (512, 0), (64, 512), (512, 120), (128, 128), (384, 128)])
def test_outputs_whose_own_rows_meet_are_refused(strides):
    assert _attn(Q, (512, 128), Q << 1, strides) == abi.DYNRAD_ERR_INVALID_ARG
    assert _read(Q, strides, Q << 1, (512, 128)) == abi.DYNRAD_ERR_INVALID_ARG
    assert _read(Q, (512, 128), Q << 1, strides) == abi.DYNRAD_ERR_INVALID_ARG
