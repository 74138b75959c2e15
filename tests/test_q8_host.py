"""Refusals of the 8-bit cache's and the selected blocks' calls that need no GPU:
the binding's, and the library's own on fake pointers; the team decode's work
split on the CPU."""

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


F16, I32 = dict(dtype=torch.float16), dict(dtype=torch.int32)
E4M3 = torch.float8_e4m3fn
T, N, H, HKV, D, NB, BS, MB, K = 5, 2, 4, 2, 64, 6, 16, 3, 2


def cache8(dtype=torch.int8):
    return torch.zeros(NB, HKV, BS, D, dtype=dtype)


def write_args():
    return dict(key=torch.zeros(T, HKV, D, **F16), value=torch.zeros(T, HKV, D, **F16), key_cache=cache8(),
                value_cache=cache8(), key_scale=torch.zeros(NB, HKV), value_scale=torch.zeros(NB, HKV),
                block_tables=torch.zeros(N, MB, **I32), context_lens=torch.ones(N, **I32),
                query_starts=torch.zeros(N + 1, **I32))


def decode_args():
    return dict(out=torch.zeros(N, H, D, **F16), query=torch.zeros(N, H, D, **F16), key_cache=cache8(),
                value_cache=cache8(), key_scale=torch.zeros(NB, HKV), value_scale=torch.zeros(NB, HKV),
                block_tables=torch.zeros(N, MB, **I32), context_lens=torch.ones(N, **I32), scale=0.125)


def selected_args():
    return dict(out=torch.zeros(N, H, D, **F16), query=torch.zeros(N, H, D, **F16),
                key_cache=torch.zeros(NB, HKV, BS, D, **F16), value_cache=torch.zeros(NB, HKV, BS, D, **F16),
                block_tables=torch.zeros(N, MB, **I32), context_lens=torch.ones(N, **I32),
                selected=torch.zeros(N, HKV, K, **I32), num_selected=torch.zeros(N, HKV, **I32), scale=0.125)


def bounds_args():
    return dict(key_bounds=torch.zeros(NB, HKV, 2, D, **F16), key_cache=torch.zeros(NB, HKV, BS, D, **F16),
                block_tables=torch.zeros(N, MB, **I32), context_lens=torch.ones(N, **I32),
                query_starts=torch.zeros(N + 1, **I32), num_tokens=T)


def select_args():
    return dict(selected=torch.zeros(N, HKV, K, **I32), num_selected=torch.zeros(N, HKV, **I32),
                query=torch.zeros(N, H, D, **F16), key_bounds=torch.zeros(NB, HKV, 2, D, **F16),
                block_tables=torch.zeros(N, MB, **I32), context_lens=torch.ones(N, **I32), block_size=BS,
                first_blocks=0, last_blocks=1)


CALLS = {"reshape_and_cache_q8": write_args, "paged_attention_decode_q8": decode_args,
         "paged_attention_decode_selected": selected_args, "block_key_bounds": bounds_args,
         "select_blocks": select_args}


@pytest.mark.parametrize("call", list(CALLS))
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA"):
        getattr(pkv, call)(**CALLS[call]())


@pytest.mark.parametrize("call", list(CALLS))
def test_every_tensor_is_checked(call):
    """Each tensor with another element type, and with another rank."""
    for name, t in CALLS[call]().items():
        if not isinstance(t, torch.Tensor):
            continue
        a = CALLS[call]()
        a[name] = t.to(torch.float64)
        with pytest.raises(TypeError, match=name):
            getattr(pkv, call)(**a)
        a = CALLS[call]()
        a[name] = t[None]
        with pytest.raises(ValueError, match="dims"):
            getattr(pkv, call)(**a)
        if name not in ("key", "value") and t.dim() > 1 and "scale" not in name:
            a = CALLS[call]()
            a[name] = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]
            with pytest.raises(ValueError, match="contiguous"):
                getattr(pkv, call)(**a)


def test_other_refusals_of_the_binding():
    a = write_args()
    a["value_cache"] = cache8(E4M3)
    with pytest.raises(TypeError, match="value_cache"):
        pkv.reshape_and_cache_q8(**a)
    for bad in (torch.zeros(T, HKV, D, **F16).transpose(0, 1).contiguous().transpose(0, 1),
                torch.zeros(T, HKV, 2 * D, **F16)[:, :, :D]):
        a = write_args()
        a["key"] = bad
        with pytest.raises(ValueError, match="contiguous"):
            pkv.reshape_and_cache_q8(**a)
    for bad in (torch.zeros(NB, HKV, 2)[:, :, 0], torch.zeros(HKV).expand(NB, HKV), torch.zeros(NB, 8)[:, :HKV]):
        for make, call in ((write_args, pkv.reshape_and_cache_q8), (decode_args, pkv.paged_attention_decode_q8)):
            a = make()
            a["key_scale"] = bad
            with pytest.raises(ValueError, match="scale|CUDA"):
                call(**a)
    a = decode_args()
    a["selected"] = torch.zeros(N, HKV, K, **I32)
    with pytest.raises(ValueError, match="together"):
        pkv.paged_attention_decode_q8(**a)
    a = bounds_args()
    a["num_tokens"] = None
    with pytest.raises(ValueError, match="together"):
        pkv.block_key_bounds(**a)
    a = bounds_args()
    a["key_scale"] = torch.zeros(NB, HKV)
    with pytest.raises(ValueError, match="key_scale"):
        pkv.block_key_bounds(**a)
    a = bounds_args()
    a["key_cache"] = cache8()
    with pytest.raises(ValueError, match="key_scale"):
        pkv.block_key_bounds(**a)


VP, ODD = ctypes.c_void_p(256), ctypes.c_void_p(264)


def refused(call, invalid, unsupported, nothing):
    for kw in nothing:
        assert call(**kw) == pkv.PKV_OK, kw
    for kw in invalid:
        assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw
    for kw in unsupported:
        assert call(**kw) == pkv.PKV_ERR_UNSUPPORTED, kw


SIZES = [dict(n=-1), dict(n=4097), dict(mb=0), dict(nb=0), dict(bs=0), dict(hkv=0), dict(mb=1 << 27), dict(nb=1 << 26),
         dict(bt=None), dict(cl=None)]
SHAPES = [dict(d=96), dict(d=256), dict(bs=12), dict(bs=256)]


def test_write_library_refuses(lib, no_gpu):
    base = dict(k=VP, ks=256, v=VP, vs=256, kc=VP, vc=VP, ksc=VP, vsc=VP, ss=4, bt=VP, mb=4, cl=VP, qs=VP, t=5, n=2, hkv=4,
                d=64, bs=16, nb=10, kind=pkv.PKV_CACHE_INT8)

    def call(**kw):
        a = dict(base, **kw)
        return lib.pkv_reshape_and_cache_q8(a["k"], a["ks"], a["v"], a["vs"], a["kc"], a["vc"], a["ksc"], a["vsc"],
                                            a["ss"], a["bt"], a["mb"], a["cl"], a["qs"], a["t"], a["n"], a["hkv"], a["d"],
                                            a["bs"], a["nb"], a["kind"], None, None)

    bad = [{name: None} for name in ("k", "v", "kc", "vc", "ksc", "vsc")] + \
          [{name: ODD} for name in ("k", "v", "kc", "vc")] + \
          [dict(t=-1), dict(ks=248), dict(ks=260), dict(vs=248), dict(ss=3), dict(kind=0), dict(kind=3), dict(qs=None)]
    refused(call, bad + SIZES, SHAPES, [dict(t=0), dict(n=0)])


def test_bounds_library_refuses(lib, no_gpu):
    base = dict(b=VP, kc=VP, ksc=None, ss=0, bt=VP, mb=4, cl=VP, qs=VP, t=5, n=2, hkv=4, d=64, bs=16, nb=10, kind=0)

    def call(**kw):
        a = dict(base, **kw)
        return lib.pkv_block_key_bounds(a["b"], a["kc"], a["ksc"], a["ss"], a["bt"], a["mb"], a["cl"], a["qs"], a["t"], a["n"],
                                        a["hkv"], a["d"], a["bs"], a["nb"], a["kind"], None, None)

    bad = [dict(b=None), dict(kc=None), dict(b=ODD), dict(kc=ODD), dict(t=-1), dict(kind=1), dict(kind=2), dict(kind=1, ksc=VP, ss=3),
           dict(kind=3), dict(kind=-1), dict(qs=None)]
    refused(call, bad + SIZES, SHAPES, [dict(t=0), dict(n=0)])


def test_decode_library_refuses(lib, no_gpu):
    base = dict(out=VP, q=VP, kc=VP, vc=VP, ksc=VP, vsc=VP, ss=5, bt=VP, mb=4, cl=VP, sel=VP, num=VP, keep=3, n=2, h=8,
                hkv=4, d=64, bs=16, nb=10, kind=pkv.PKV_CACHE_E4M3, scale=0.125, ctas=3, ws=VP, wsb=1 << 40)

    def q8(**kw):
        a = dict(base, **kw)
        return lib.pkv_paged_attention_decode_q8(
            a["out"], a["q"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["ss"], a["bt"], a["mb"], a["cl"], a["sel"], a["num"],
            a["keep"], a["n"], a["h"], a["hkv"], a["d"], a["bs"], a["nb"], a["kind"], ctypes.c_float(a["scale"]),
            a["ctas"], a["ws"], a["wsb"], None, None)

    def f16(**kw):
        a = dict(base, **kw)
        return lib.pkv_paged_attention_decode_selected(
            a["out"], a["q"], a["kc"], a["vc"], a["bt"], a["mb"], a["cl"], a["sel"], a["num"], a["keep"], a["n"],
            a["h"], a["hkv"], a["d"], a["bs"], a["nb"], ctypes.c_float(a["scale"]), a["ctas"], a["ws"], a["wsb"],
            None, None)

    bad = [{name: None} for name in ("out", "q", "kc", "vc", "sel", "num", "ws")] + \
          [{name: ODD} for name in ("out", "q", "kc", "vc", "ws")] + SIZES + \
          [dict(keep=0), dict(keep=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
           dict(scale=-1.0), dict(ctas=-1), dict(ctas=4097), dict(wsb=100), dict(h=6), dict(h=0)]
    shapes = SHAPES + [dict(h=68)]
    refused(q8, bad + [dict(ksc=None), dict(vsc=None), dict(ss=3), dict(kind=0), dict(kind=3)], shapes, [dict(n=0)])
    refused(f16, bad + [dict(sel=None, num=None)], shapes, [dict(n=0)])


def test_select_library_refuses(lib, no_gpu):
    base = dict(sel=VP, num=VP, q=VP, b=VP, bt=VP, mb=4, cl=VP, n=2, h=8, hkv=4, d=64, bs=16, nb=10, keep=3, first=1,
                last=2, ws=VP, wsb=1 << 40)

    def call(**kw):
        a = dict(base, **kw)
        return lib.pkv_select_blocks(a["sel"], a["num"], a["q"], a["b"], a["bt"], a["mb"], a["cl"], a["n"], a["h"],
                                     a["hkv"], a["d"], a["bs"], a["nb"], a["keep"], a["first"], a["last"], a["ws"],
                                     a["wsb"], None, None)

    bad = [{name: None} for name in ("sel", "num", "q", "b", "ws")] + [{name: ODD} for name in ("q", "b", "ws")] + \
          SIZES + [dict(keep=0), dict(first=-1), dict(last=-1), dict(first=2), dict(last=3), dict(wsb=100), dict(h=6),
                   dict(h=0)]
    refused(call, bad, SHAPES + [dict(h=68)], [dict(n=0)])


def test_workspace_sizes(lib, no_gpu):
    size = lib.pkv_decode_team_workspace_size
    assert size(8, 2, 128, 4) > 0
    assert size(8, 3, 128, 4) == size(34, 2, 128, 4) == size(8, 2, 96, 4) == size(8, 2, 128, -1) == 0
    assert size(8, 2, 128, 4097) == 0
    size = lib.pkv_select_workspace_size
    assert size(2, 4, 100) >= 2 * 4 * 100 * 12
    assert size(-1, 4, 100) == size(4097, 4, 100) == size(2, 0, 100) == size(2, 4, 0) == 0


def test_team_schedule(tmp_path):
    """The work split's host check (tests/cpp/test_team_schedule.cpp)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "test_team_schedule"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", os.path.join(root, "paged_kv_cache_152_gb300", "csrc"),
                    os.path.join(root, "tests", "cpp", "test_team_schedule.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "team schedule ok" in r.stdout


def test_scratch_is_given_back():
    """A call's scratch goes back to the allocator, of the call's stream, whether
    the library takes the call, refuses it or ctypes does."""
    class Allocator:
        def __init__(self):
            self.out, self.asked = set(), []

        def _cuda_cudaCachingAllocator_raw_alloc(self, size, stream):
            self.asked.append((size, stream))
            self.out.add(512 * len(self.asked))
            return 512 * len(self.asked)

        def _cuda_cudaCachingAllocator_raw_delete(self, address):
            self.out.remove(address)

    raw, seen = Allocator(), []

    def call(*args):
        assert raw.out == {args[2]}
        seen.append(args)
        if args[0] == "raise":
            raise TypeError("argument 1")
        return args[0]

    assert pkv._call_with_bytes(raw, call, (0, 7), 4096, 99, 5) == 0
    assert pkv._call_with_bytes(raw, call, (3, 7), 256, None, 6) == 3
    with pytest.raises(TypeError):
        pkv._call_with_bytes(raw, call, ("raise", 7), 256, None, 6)
    assert seen == [(0, 7, 512, 4096, 99, 5), (3, 7, 1024, 256, None, 6), ("raise", 7, 1536, 256, None, 6)]
    assert raw.asked == [(4096, 5), (256, 6), (256, 6)] and not raw.out
