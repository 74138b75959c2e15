"""GPU checks of the chunk attention's bounded waits: how long they take to give
up, and that a kernel which gave up in mid-work leaves the device as it was.

Every wait here ends by itself: the limits are the kernel's own or shorter.
"""

import ctypes

import numpy as np
import pytest
import torch

from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from paged_kv_cache_152_gb300 import build
    build.build()
    import paged_kv_cache_152_gb300 as m
    m.load()
    return m


def test_both_waits_have_the_limit_they_state(pkv):
    """A second and more each, and no more than a few: neither gives up while
    the other, which it may depend on, still waits in good order."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    elapsed = torch.zeros(2, dtype=torch.int64, device="cuda")
    pkv.selftest_chunk_waits(status, elapsed)
    torch.cuda.synchronize()
    assert int(status.item()) == pkv.PKV_ERR_DEVICE_TIMEOUT
    barrier, counter = (x * 1e-9 for x in elapsed.tolist())
    assert 0.5 <= barrier <= 5.0 and 0.5 <= counter <= 5.0, (barrier, counter)


CASES = [
    dict(h=8, hkv=2, d=128, bs=16, seqs=[(1, 3000), (70, 500), (200, 210), (0, 9), (3, 0)]),
    dict(h=4, hkv=4, d=64, bs=16, seqs=[(300, 1900), (1, 2500), (129, 700)]),
    dict(h=8, hkv=1, d=128, bs=32, seqs=[(260, 2300), (90, 1700)], window=1000),
    dict(h=2, hkv=2, d=128, bs=128, seqs=[(700, 900)], causal=False),
]


@pytest.mark.parametrize("k", range(len(CASES)))
@pytest.mark.parametrize("num_ctas", [0, 3])
def test_giving_up_in_mid_work(pkv, k, num_ctas):
    """With a limit of no try, some wait of every call gives up; with a few,
    calls end in every stage of their work.  The status says so, rows of no
    sequence stay, and a call behind it has its usual bits."""
    c = Case(30 + k, before=1, behind=2, **CASES[k]).gpu()
    good = c.call(pkv, num_ctas=num_ctas).clone()
    c.check(good)
    t, lib = c.t, pkv.load()
    (rows, h, d), (nb, hkv, bs, _), (n, mb) = t["q"].shape, t["kc"].shape, t["tables"].shape
    ws = pkv.new_chunk_workspace(rows, h, hkv, d, num_ctas)
    ws.fill_(0)
    codes = []
    for tries in (0, 0, 1, 2, 3, 4, 6, 8, 12, 20, 1 << 19):
        out = torch.full_like(c.out, -77.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        rc = lib.pkv_selftest_chunk_give_up(
            out.data_ptr(), t["q"].data_ptr(), t["kc"].data_ptr(), t["vc"].data_ptr(), t["tables"].data_ptr(), mb,
            t["lens"].data_ptr(), t["starts"].data_ptr(), rows, n, h, hkv, d, bs, nb, ctypes.c_float(c.scale),
            int(c.causal), c.window, num_ctas, ws.data_ptr(), ws.numel(), status.data_ptr(),
            torch.cuda.current_stream().cuda_stream, tries)
        assert rc == pkv.PKV_OK
        torch.cuda.synchronize()
        codes.append(int(status.item()))
        assert codes[-1] in (pkv.PKV_OK, pkv.PKV_ERR_DEVICE_TIMEOUT)
        assert (out[:1] == -77.0).all() and (out[rows - 2:] == -77.0).all()
        if codes[-1] == pkv.PKV_OK:
            assert torch.equal(out, good)
        again = c.call(pkv, out=torch.full_like(c.out, -77.0), num_ctas=num_ctas, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(again, good) and int(c.status.item()) == 0
    assert codes[0] == codes[1] == pkv.PKV_ERR_DEVICE_TIMEOUT and codes[-1] == pkv.PKV_OK
