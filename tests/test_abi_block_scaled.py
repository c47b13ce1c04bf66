"""The block-scaled cache's calls without a GPU: bad arguments are refused on the host before any launch."""
import ctypes
import os
import re

import pytest
import torch

import paged_kv_cache_185_gb300 as wllm
from paged_kv_cache_185_gb300 import binding, build
from tests.test_abi import desc
from tests.test_waits_source import waits

BF, F16, F32, U8, I32, I64 = torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.int32, torch.int64
INVALID, UNSUPPORTED = binding.WLLM_ERR_INVALID_ARG, binding.WLLM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def call(lib, name, a, names, *scalars):
    n = lib.wllm_launch_count()
    rc = getattr(lib, name)(*[None if a[x] is None else ctypes.byref(a[x]) for x in names], *scalars, None)
    assert lib.wllm_launch_count() == n and (rc == 0 or lib.wllm_last_error())
    return rc


def at(i):
    return 0x1000000 * (i + 1)


def slots(lib, change=(), B=3, T=8, F=10, M=4, bs=16):
    names = ("slots", "pos", "starts", "lens_out", "free_out", "bt", "lens", "new", "free", "count")
    a = dict(slots=desc((T,), I64, data=at(0)), pos=desc((T,), I64, data=at(1)), starts=desc((B + 1,), I32, data=at(2)),
             lens_out=desc((B,), I32, data=at(3)), free_out=desc((1,), I32, data=at(4)), bt=desc((B, M), I32, data=at(5)),
             lens=desc((B,), I32, data=at(6)), new=desc((B,), I32, data=at(7)), free=desc((F,), I32, data=at(8)),
             count=desc((1,), I32, data=at(9)))
    a.update(change)
    return call(lib, "wllm_assign_slots", a, names, bs)


@pytest.mark.parametrize("change", [
    dict(slots=desc((8,), I32, data=at(0))), dict(slots=desc((8,), I64, stride=(2,), data=at(0))), dict(slots=None),
    dict(pos=desc((7,), I64, data=at(1))), dict(pos=desc((8,), I32, data=at(1))), dict(starts=desc((3,), I32, data=at(2))),
    dict(starts=desc((4,), I64, data=at(2))), dict(lens_out=desc((4,), I32, data=at(3))), dict(free_out=desc((2,), I32, data=at(4))),
    dict(free_out=None), dict(bt=desc((3, 4), I64, data=at(5))), dict(bt=desc((3, 4), I32, stride=(8, 2), data=at(5))),
    dict(bt=desc((3, 4), I32, stride=(2, 1), data=at(5))),                                   # rows that overlap
    dict(lens=desc((2,), I32, data=at(6))), dict(new=desc((3,), I64, data=at(7))), dict(new=desc((3,), I32, stride=(2,), data=at(7))),
    dict(free=desc((10,), I64, data=at(8))), dict(free=desc((2, 5), I32, data=at(8))), dict(count=desc((1,), I64, data=at(9))),
    dict(lens_out=desc((3,), I32, data=at(6) + 4)),                                          # in place, but shifted
    dict(pos=desc((8,), I64, data=at(0))), dict(free=desc((10,), I32, data=at(5) + 8)), dict(new=desc((3,), I32, data=at(3))),
    dict(starts=desc((4,), I32, data=at(7) + 8)), dict(count=desc((1,), I32, data=at(8) + 36)),
    dict(slots=desc((8,), I64, data=at(0) + 4)), dict(lens=desc((3,), I32, data=at(6) + 2)), dict(bt=desc((3, 4), I32, data=at(5) + 1))])
def test_slots_refuses(lib, change):
    assert slots(lib, change) == INVALID


def test_slots_refuses_sizes(lib):
    assert slots(lib, bs=12) == UNSUPPORTED
    assert slots(lib, bs=0) == UNSUPPORTED
    assert slots(lib, B=16385) == UNSUPPORTED
    assert slots(lib, M=2 ** 28) == UNSUPPORTED


def append(lib, change=(), T=6, B=3, Hkv=2, D=128, bs=16, dt=BF, starts=True, size=None):
    names = ("key", "value", "kc", "vc", "ks", "vs", "bt", "cl", "qsl")
    a = dict(key=desc((T, Hkv, D), dt), value=desc((T, Hkv, D), dt), kc=desc((8, Hkv, bs, D), U8), vc=desc((8, Hkv, bs, D), U8),
             ks=desc((8, Hkv), F32), vs=desc((8, Hkv), F32), bt=desc((B, 4), I32), cl=desc((B,), I32),
             qsl=desc((B + 1,), I32) if starts else None)
    a.update(change)
    return call(lib, "wllm_reshape_and_cache_block_scaled", a, names, size or bs)


CACHE = [dict(kc=desc((8, 2, 16, 128), BF)), dict(vc=desc((7, 2, 16, 128), U8)), dict(kc=desc((8, 2, 16, 128), U8, data=0x10008)),
         dict(kc=desc((8, 2, 16, 128), U8, stride=(8192, 4096, 256, 1)), vc=desc((8, 2, 16, 128), U8)), dict(ks=desc((8, 2), F16)),
         dict(ks=desc((8, 3), F32)), dict(vs=desc((7, 2), F32)), dict(vs=desc((8, 2), F32, stride=(4, 1))), dict(ks=None),
         dict(vs=desc((16,), F32)), dict(bt=desc((3, 4), I64)), dict(bt=desc((2, 4), I32)), dict(bt=desc((3, 4), I32, stride=(8, 2))),
         dict(cl=desc((3,), I64)), dict(cl=desc((3,), I32, stride=(2,))), dict(ks=desc((8, 2), F32, data=0x10002)),
         dict(cl=desc((3,), I32, data=0x10002)), dict(bt=desc((3, 4), I32, data=0x10001))]


@pytest.mark.parametrize("change", CACHE + [
    dict(key=desc((6, 256), BF)), dict(key=desc((6, 2, 128), I32)), dict(value=desc((6, 2, 128), F16)), dict(value=desc((5, 2, 128), BF)),
    dict(key=desc((6, 2, 128), BF, stride=(512, 256, 2))), dict(key=desc((6, 2, 64), BF), value=desc((6, 2, 64), BF)),
    dict(key=desc((6, 3, 128), BF), value=desc((6, 3, 128), BF)), dict(key=desc((6, 2, 128), BF, data=0x10001)),
    dict(qsl=desc((3,), I32)), dict(qsl=desc((4,), I64)), dict(qsl=desc((4,), I32, stride=(2,))), dict(qsl=None)])
def test_append_refuses(lib, change):
    assert append(lib, change) == INVALID


def test_append_refuses_sizes(lib):
    assert append(lib, size=32) == INVALID
    assert append(lib, D=96) == UNSUPPORTED
    assert append(lib, D=512) == UNSUPPORTED
    assert append(lib, bs=4) == UNSUPPORTED
    assert append(lib, bs=24) == UNSUPPORTED
    assert append(lib, bs=512) == UNSUPPORTED
    assert append(lib, T=2, starts=False) == INVALID  # a row a sequence
    assert append(lib, T=0) == 0
    assert append(lib, T=0, B=0) == 0
    assert append(lib, T=0, B=0, starts=False) == 0
    assert append(lib, dict(kc=desc((0, 2, 16, 128), U8, data=None), vc=desc((0, 2, 16, 128), U8, data=None),
                            ks=desc((0, 2), F32, data=None), vs=desc((0, 2), F32, data=None))) == INVALID


def attention(lib, kind, change=(), B=3, T=None, Hq=4, Hkv=2, D=128, bs=16, dt=BF, scale=0.1, heads=None, size=None):
    T = (B if kind == "decode" else 7) if T is None else T
    names = ("out", "q", "kc", "vc", "ks", "vs", "bt", "cl") + (("ws",) if kind == "decode" else ("qsl", "ws"))
    a = dict(out=desc((T, Hq, D), dt), q=desc((T, Hq, D), dt), kc=desc((8, Hkv, bs, D), U8), vc=desc((8, Hkv, bs, D), U8),
             ks=desc((8, Hkv), F32), vs=desc((8, Hkv), F32), bt=desc((B, 4), I32), cl=desc((B,), I32), qsl=desc((B + 1,), I32),
             ws=desc((1 << 26,), U8, data=0x40000000))
    a.update(change)
    return call(lib, f"wllm_paged_attention_{kind}_block_scaled", a, names, heads or Hkv, scale, size or bs)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("change", CACHE + [
    dict(q=desc((3, 512), BF)), dict(q=desc((3, 4, 128), F32), out=desc((3, 4, 128), F32)), dict(out=desc((3, 4, 128), F16)),
    dict(out=desc((3, 4, 64), BF)), dict(q=desc((3, 4, 128), BF, stride=(1024, 256, 2)), out=desc((3, 4, 128), BF)),
    dict(q=desc((3, 4, 64), BF), out=desc((3, 4, 64), BF)), dict(q=desc((3, 5, 128), BF), out=desc((3, 5, 128), BF)),
    dict(q=desc((3, 4, 128), BF, data=0x10001), out=desc((3, 4, 128), BF)), dict(out=None), dict(cl=None)])
def test_attention_refuses(lib, kind, change):
    assert attention(lib, kind, change, T=3) == INVALID


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_attention_refuses_sizes(lib, kind):
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert attention(lib, kind, scale=scale) == INVALID
    assert attention(lib, kind, heads=3) == INVALID
    assert attention(lib, kind, size=32) == INVALID
    assert attention(lib, kind, D=96) == UNSUPPORTED
    assert attention(lib, kind, D=512) == UNSUPPORTED
    assert attention(lib, kind, bs=4) == UNSUPPORTED
    assert attention(lib, kind, dict(kc=desc((0, 2, 16, 128), U8, data=None), vc=desc((0, 2, 16, 128), U8, data=None),
                                     ks=desc((0, 2), F32, data=None), vs=desc((0, 2), F32, data=None))) == INVALID
    assert attention(lib, kind, B=0, T=0) == 0
    assert attention(lib, kind, Hq=0) == 0


def test_prefill_refuses(lib):
    assert attention(lib, "prefill", D=256) == UNSUPPORTED
    assert attention(lib, "prefill", dict(qsl=desc((3,), I32))) == INVALID
    assert attention(lib, "prefill", dict(qsl=desc((4,), I64))) == INVALID
    assert attention(lib, "prefill", dict(qsl=None)) == INVALID
    assert attention(lib, "prefill", T=0) == 0


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_attention_refuses_workspaces(lib, kind):
    assert attention(lib, kind, dict(ws=None)) == INVALID
    assert attention(lib, kind, dict(ws=desc((1 << 25, 2), U8))) == INVALID
    assert attention(lib, kind, dict(ws=desc((1 << 25,), U8, data=None))) == INVALID


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_attention_refuses_half_boxes(lib, kind):
    assert attention(lib, kind, D=64, bs=8) == UNSUPPORTED


def test_binding_refuses():
    x, c = torch.zeros(2, 2, 64, dtype=BF), torch.zeros(3, 2, 16, 64, dtype=U8)
    s, i, l = torch.zeros(3, 2), torch.zeros(2, dtype=I32), torch.zeros(2, dtype=I64)
    with pytest.raises(ValueError, match="CUDA"):
        wllm.assign_slots(l, i, i[:, None], i, i, i, i[:1], 16)
    with pytest.raises(ValueError, match="CUDA"):
        wllm.reshape_and_cache_block_scaled(x, x, c, c, s, s, i[:, None], i, 16)
    with pytest.raises(ValueError, match="CUDA"):
        wllm.paged_attention_decode_block_scaled(x, x, c, c, s, s, i[:, None], i, 2, 0.1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        wllm.paged_attention_prefill_block_scaled(x, x, c, c, s, s, i[:, None], i, i, 2, 0.1, 16)


FILES = ["assign_slots.cu", "append_block_scaled.cu", "decode_block_scaled.cu", "prefill_block_scaled.cu"]


@pytest.mark.parametrize("name", FILES)
def test_kernels_read_what_others_write_by_plain_loads(name):
    """Dependent launches are alive while the kernel before them writes: no non-coherent loads."""
    code = re.sub(r"//.*", "", open(os.path.join(build.CSRC, name)).read())
    assert "launch_dependent(" in code and "grid_wait()" in code
    assert not re.search(r"__ldg|__ldcs|ld\.global\.nc|\b__restrict__", code)


@pytest.mark.parametrize("name", FILES)
def test_no_lane_gives_up_alone(name):
    """One lane waits for its warp and tells it, the warp votes, or only copies in flight are let land."""
    for number, code in waits(os.path.join(build.CSRC, name)):
        assert re.match(r"(for \(.*\) mbar_wait_bounded\(|(if \(lane == 0\) |const bool )?(got|ok) = mbar_wait_bounded\()", code), f"{name}:{number}: {code}"
