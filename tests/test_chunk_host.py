"""Refusals of the chunk attention and of the norm with rotation that need no
GPU: the binding's, and the library's own on fake pointers."""

import ctypes
import os
import subprocess

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
    """Fake device pointers must be rejected before any launch; never run them
    where a launch could reach a GPU."""
    if torch.cuda.is_available():
        pytest.skip("fake-pointer host checks run on GPU-less hosts only")


F16 = dict(dtype=torch.float16)


def chunk_args(t=5, h=4, hkv=2, d=64, nb=6, bs=16, n=2, mb=3):
    return dict(out=torch.zeros(t, h, d, **F16), query=torch.zeros(t, h, d, **F16),
                key_cache=torch.zeros(nb, hkv, bs, d, **F16), value_cache=torch.zeros(nb, hkv, bs, d, **F16),
                block_tables=torch.zeros(n, mb, dtype=torch.int32), context_lens=torch.ones(n, dtype=torch.int32),
                query_starts=torch.zeros(n + 1, dtype=torch.int32), scale=d ** -0.5)


@pytest.mark.parametrize("name,bad,error,match", [
    ("query", torch.zeros(5, 4, 64), TypeError, "query"),
    ("query", torch.zeros(5, 4, 64, dtype=torch.bfloat16), TypeError, "query"),
    ("query", torch.zeros(4, 5, 64, **F16).transpose(0, 1), ValueError, "contiguous"),
    ("query_starts", torch.zeros(3, dtype=torch.int64), TypeError, "query_starts"),
    ("query_starts", torch.zeros(1, 3, dtype=torch.int32), ValueError, "dims"),
    ("block_tables", torch.zeros(2, 3, dtype=torch.int64), TypeError, "block_tables"),
    ("context_lens", torch.ones(2, dtype=torch.int64), TypeError, "context_lens"),
    ("out", torch.zeros(5, 4, 64), TypeError, "out"),
    ("out", torch.zeros(5, 4, 64, **F16), ValueError, "CUDA"),
])
def test_chunk_binding_refuses(name, bad, error, match):
    a = chunk_args()
    a[name] = bad
    with pytest.raises(error, match=match):
        pkv.paged_attention_chunk(**a)


def test_chunk_library_refuses(lib, no_gpu):
    vp, odd = ctypes.c_void_p(256), ctypes.c_void_p(264)
    base = dict(out=vp, q=vp, kc=vp, vc=vp, bt=vp, mb=4, cl=vp, qs=vp, t=5, n=2, h=8, hkv=4, d=64, bs=16, nb=10,
                scale=0.125, causal=1, window=0, ctas=3, ws=vp, wsb=1 << 40)

    def call(**kw):
        a = dict(base, **kw)
        return lib.pkv_paged_attention_chunk(
            a["out"], a["q"], a["kc"], a["vc"], a["bt"], a["mb"], a["cl"], a["qs"], a["t"], a["n"], a["h"], a["hkv"],
            a["d"], a["bs"], a["nb"], ctypes.c_float(a["scale"]), a["causal"], a["window"], a["ctas"], a["ws"],
            a["wsb"], None, None)

    assert call(t=0) == call(n=0) == pkv.PKV_OK
    for name in ("out", "q", "kc", "vc", "bt", "cl", "qs", "ws"):
        assert call(**{name: None}) == pkv.PKV_ERR_INVALID_ARG, name
    for name in ("out", "q", "kc", "vc", "ws"):
        assert call(**{name: odd}) == pkv.PKV_ERR_INVALID_ARG, name
    for kw in (dict(t=-1), dict(n=-1), dict(n=4097), dict(mb=0), dict(nb=0), dict(ctas=-1), dict(ctas=4097),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(window=-1), dict(causal=0, window=4), dict(h=6), dict(h=0), dict(hkv=0), dict(bs=0),
               dict(mb=1 << 27), dict(nb=1 << 26), dict(wsb=100)):
        assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw
    for kw in (dict(d=96), dict(d=256), dict(bs=12), dict(bs=256), dict(h=68)):
        assert call(**kw) == pkv.PKV_ERR_UNSUPPORTED, kw


def test_chunk_workspace_sizes(lib, no_gpu):
    size = lib.pkv_chunk_workspace_size
    assert size(100, 8, 2, 128, 4) > 0
    assert size(100, 8, 3, 128, 4) == size(100, 68, 4, 128, 4) == size(100, 8, 2, 96, 4) == 0
    assert size(-1, 8, 2, 128, 4) == size(100, 8, 2, 128, -1) == size(100, 8, 2, 128, 4097) == 0


def test_chunk_schedule(tmp_path):
    """The work split's host check (tests/cpp/test_chunk_schedule.cpp)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "test_chunk_schedule"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", os.path.join(root, "paged_kv_cache_152_gb300", "csrc"),
                    os.path.join(root, "tests", "cpp", "test_chunk_schedule.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "chunk schedule ok" in r.stdout


def rope_args(t=3, h=4, hkv=2, d=64, rot=64):
    return dict(query_out=torch.zeros(t, h, d, **F16), key_out=torch.zeros(t, hkv, d, **F16),
                query=torch.zeros(t, h, d, **F16), key=torch.zeros(t, hkv, d, **F16),
                positions=torch.zeros(t, dtype=torch.int64), cos_sin=torch.zeros(8, rot))


def test_rope_binding_refuses():
    with pytest.raises(ValueError, match="CUDA"):
        pkv.qk_norm_rope(**rope_args())
    for name, bad, error, match in (
            ("query", torch.zeros(3, 4, 64), TypeError, "query"),
            ("query", torch.zeros(3, 64, 4, **F16).transpose(1, 2), ValueError, "contiguous"),
            ("query", torch.zeros(3, 4, 128, **F16)[:, :, :64], ValueError, "contiguous"),
            ("query", torch.zeros(1, 4, 64, **F16).expand(3, 4, 64), ValueError, "overlap"),
            ("query", torch.zeros(3, 4 * 64 + 4, **F16)[:, :256].view(3, 4, 64), ValueError, "multiple of 8"),
            ("key", torch.zeros(3, 2, 64, dtype=torch.bfloat16), TypeError, "key"),
            ("query_out", torch.zeros(3, 256, **F16), ValueError, "dims")):
        a = rope_args()
        a[name] = bad
        with pytest.raises(error, match=match):
            pkv.qk_norm_rope(**a)


def test_rope_library_refuses(lib, no_gpu):
    vp, odd = ctypes.c_void_p(256), ctypes.c_void_p(264)
    base = dict(qo=vp, qos=256, ko=vp, kos=128, q=vp, qs=256, k=vp, ks=128, v=vp, vs=128, kc=vp, vc=vp, sm=vp, pos=vp,
                cs=vp, maxp=10, rot=64, inter=0, wq=vp, wk=vp, eps=1e-6, t=3, h=4, hkv=2, d=64, bs=16, nb=4)

    def plain(**kw):
        a = dict(base, **kw)
        return lib.pkv_qk_norm_rope(a["qo"], a["qos"], a["ko"], a["kos"], a["q"], a["qs"], a["k"], a["ks"], a["pos"],
                                    a["cs"], a["maxp"], a["rot"], a["inter"], a["wq"], a["wk"],
                                    ctypes.c_float(a["eps"]), a["t"], a["h"], a["hkv"], a["d"], None, None)

    def cached(**kw):
        a = dict(base, **kw)
        return lib.pkv_qk_norm_rope_and_cache(
            a["qo"], a["qos"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["kc"], a["vc"], a["sm"], a["pos"],
            a["cs"], a["maxp"], a["rot"], a["inter"], a["wq"], a["wk"], ctypes.c_float(a["eps"]), a["t"], a["h"],
            a["hkv"], a["d"], a["bs"], a["nb"], None, None)

    both = [dict(qo=None), dict(q=None), dict(k=None), dict(qo=odd), dict(q=odd), dict(k=odd), dict(pos=None),
            dict(cs=None), dict(cs=odd), dict(maxp=0), dict(wq=odd), dict(wk=odd), dict(qos=248), dict(qs=260),
            dict(ks=120), dict(rot=8), dict(rot=24), dict(rot=80), dict(rot=-16), dict(eps=-1.0),
            dict(eps=float("nan")), dict(eps=float("inf")), dict(t=-1), dict(h=0), dict(hkv=0), dict(d=0),
            dict(d=60)]
    for call, more in ((plain, [dict(ko=None), dict(ko=odd), dict(kos=120)]),
                       (cached, [dict(v=None), dict(kc=None), dict(vc=None), dict(sm=None), dict(v=odd), dict(kc=odd),
                                 dict(vc=odd), dict(vs=120), dict(bs=0), dict(nb=0)])):
        assert call(t=0) == pkv.PKV_OK
        for kw in both + more:
            assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw
        assert call(d=264, qs=8192, ks=8192, vs=8192, qos=8192, kos=8192) == pkv.PKV_ERR_UNSUPPORTED
