"""Refusals of the chunk attention's self-tests that need no GPU."""

import ctypes

import pytest
import torch

import paged_kv_cache_152_gb300 as pkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_kv_cache_152_gb300 import build
    build.build()
    return pkv.load()


@pytest.fixture
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("fake-pointer host checks run on GPU-less hosts only")


def test_waits_need_device_words(lib, no_gpu):
    vp = ctypes.c_void_p(256)
    assert lib.pkv_selftest_chunk_waits(None, vp, None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_selftest_chunk_waits(vp, None, None) == pkv.PKV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        pkv.selftest_chunk_waits(None, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        pkv.selftest_chunk_waits(torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int64))


def test_give_up_refuses_what_the_call_refuses(lib, no_gpu):
    vp = ctypes.c_void_p(256)

    def call(tries=0, t=5, scale=0.125, ws=vp):
        return lib.pkv_selftest_chunk_give_up(vp, vp, vp, vp, vp, 4, vp, vp, t, 2, 8, 4, 64, 16, 10,
                                              ctypes.c_float(scale), 1, 0, 3, ws, 1 << 40, None, None, tries)

    assert call(t=0) == pkv.PKV_OK
    assert call(tries=-1) == call(tries=(1 << 19) + 1) == pkv.PKV_ERR_INVALID_ARG
    assert call(scale=-1.0) == call(ws=None) == pkv.PKV_ERR_INVALID_ARG
