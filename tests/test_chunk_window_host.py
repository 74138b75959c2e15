"""The chunk attention's window as the library receives it (no GPU)."""

import ctypes
import sys

import pytest
import torch

import paged_kv_cache_152_gb300 as pkv


@pytest.mark.parametrize("window", [0, 1, 4096, (1 << 30) - 1, (1 << 31) - 1, 1 << 31, (1 << 32) + 5, sys.maxsize, -1,
                                    -(1 << 32) + 5])
def test_any_window_arrives_as_what_it_means(monkeypatch, window):
    """No context is longer than 2^30: a longer window hides nothing, however
    large the number, and a negative one stays negative (refused)."""
    seen = []
    monkeypatch.setattr(pkv, "_checked", lambda specs: 0)
    monkeypatch.setattr(pkv, "_launch", lambda fn, what, index, stream, args: seen.append(args))
    f16, i32 = torch.float16, torch.int32
    out = torch.zeros(5, 4, 64, dtype=f16)
    pool = torch.zeros(6, 2, 16, 64, dtype=f16)
    pkv.paged_attention_chunk(out, out.clone(), pool, pool.clone(), torch.zeros(2, 3, dtype=i32), torch.ones(2, dtype=i32),
                              torch.zeros(3, dtype=i32), 0.125, window=window,
                              workspace=torch.zeros(256, dtype=torch.uint8))
    types = pkv.SIGNATURES["pkv_paged_attention_chunk"][1]
    at = 17
    assert types[at] is ctypes.c_int and seen[0][at - 1] == 1
    arrived = ctypes.c_int(seen[0][at]).value
    assert arrived == window if -1 <= window < 1 << 31 else arrived < 0 if window < 0 else arrived >= 1 << 30
