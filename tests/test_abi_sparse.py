"""The rotary append and block-sparse decode without a GPU: bad arguments are refused on the host before any launch."""
import ctypes

import pytest
import torch

import paged_kv_cache_185_gb300 as wllm
from paged_kv_cache_185_gb300 import binding, build
from tests.test_abi import desc

BF, F16, F32, U8, I32, I64 = torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.int32, torch.int64
INVALID, UNSUPPORTED = binding.WLLM_ERR_INVALID_ARG, binding.WLLM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def refs(a, names):
    return [None if a[n] is None else ctypes.byref(a[n]) for n in names]


def rotary(style=0, axes=1, sections=(), eps=1e-6):
    how = binding.WllmRotary(style, axes)
    how.sections[:len(sections)] = sections
    how.eps = eps
    return how


ROTATE = ("q_out", "q", "key", "value", "k_cache", "v_cache", "slots", "positions", "cos_sin", "q_weight", "k_weight")


def rotate(lib, change=(), scales=None, how=None, T=6, Hq=4, Hkv=2, D=64, R=64, bs=16, dt=BF, cache=None):
    c = cache or dt
    a = dict(q_out=desc((T, Hq, D), dt, data=0x900000), q=desc((T, Hq, D), dt), key=desc((T, Hkv, D), dt),
             value=desc((T, Hkv, D), dt), k_cache=desc((8, Hkv, bs, D), c), v_cache=desc((8, Hkv, bs, D), c),
             slots=desc((T,), I64), positions=desc((T,), I32), cos_sin=desc((100, R), F32), q_weight=desc((D,), dt),
             k_weight=desc((D,), dt))
    a.update(change)
    how = rotary() if how is None else how
    tail = [] if scales is None else list(scales)
    f = lib.wllm_rotate_and_cache if scales is None else lib.wllm_rotate_and_cache_fp8
    n = lib.wllm_launch_count()
    rc = f(*refs(a, ROTATE), None if how == "none" else ctypes.byref(how), *tail, None)
    assert lib.wllm_launch_count() == n and (rc == 0 or lib.wllm_last_error())
    return rc


@pytest.mark.parametrize("change,status", [
    (dict(q=desc((6, 256), BF)), INVALID),                                      # rank
    (dict(q=None), INVALID),
    (dict(positions=None), INVALID),
    (dict(key=desc((6, 2, 64), F16)), INVALID),                                 # one type
    (dict(q_out=desc((6, 4, 64), F32)), INVALID),
    (dict(k_cache=desc((8, 2, 16, 64), F16)), INVALID),
    (dict(k_cache=desc((8, 3, 16, 64), BF), v_cache=desc((8, 3, 16, 64), BF)), INVALID),
    (dict(key=desc((5, 2, 64), BF), value=desc((5, 2, 64), BF)), INVALID),      # another T
    (dict(value=desc((6, 3, 64), BF)), INVALID),
    (dict(slots=desc((5,), I64)), INVALID),
    (dict(slots=desc((6,), F32)), INVALID),
    (dict(slots=desc((6,), I64, stride=(2,))), INVALID),
    (dict(positions=desc((7,), I32)), INVALID),
    (dict(positions=desc((2, 6), I32)), INVALID),                               # two axes, one named
    (dict(positions=desc((6,), F32)), INVALID),
    (dict(positions=desc((6,), I32, stride=(2,))), INVALID),
    (dict(cos_sin=desc((100, 64), F16)), INVALID),
    (dict(cos_sin=desc((100, 64), F32, stride=(128, 2))), INVALID),
    (dict(cos_sin=desc((100, 80), F32)), INVALID),                              # more than head_dim
    (dict(cos_sin=desc((100, 24), F32)), UNSUPPORTED),
    (dict(q_weight=desc((32,), BF)), INVALID),
    (dict(q_weight=desc((64,), F16)), INVALID),
    (dict(q_weight=desc((64,), F32)), INVALID),                                 # two weights, two types
    (dict(k_weight=desc((64,), BF, stride=(2,))), INVALID),
    (dict(k_weight=desc((64,), BF, data=0x10001)), INVALID),
    (dict(q=desc((6, 4, 64), BF, stride=(512, 128, 2))), INVALID),
    (dict(q_out=desc((6, 4, 64), BF, data=0x10040)), INVALID),                  # overlaps q, is not q
    (dict(q_out=desc((6, 4, 64), BF, stride=(512, 64, 1))), INVALID),           # q's memory in another order
    (dict(q=desc((6, 4, 64), BF, data=0x10001)), INVALID),                      # half an element
    (dict(k_cache=desc((8, 2, 16, 64), BF, stride=(2048, 1024, 128, 1))), INVALID),
])
def test_rotate_refuses(lib, change, status):
    assert rotate(lib, change) == status


def test_rotate_refuses_options_and_sizes(lib):
    two = dict(positions=desc((2, 6), I32))
    assert rotate(lib, how="none") == INVALID
    assert rotate(lib, how=rotary(style=2)) == INVALID
    assert rotate(lib, how=rotary(axes=0)) == INVALID
    assert rotate(lib, how=rotary(axes=5)) == INVALID
    assert rotate(lib, how=rotary(eps=-1.0)) == INVALID
    assert rotate(lib, how=rotary(eps=float("nan"))) == INVALID
    assert rotate(lib, two, how=rotary(axes=2, sections=(8, 16))) == INVALID    # 24 of 32 pairs
    assert rotate(lib, two, how=rotary(axes=2, sections=(40, -8))) == INVALID
    assert rotate(lib, D=72, R=64) == UNSUPPORTED
    assert rotate(lib, D=272, R=64) == UNSUPPORTED
    assert rotate(lib, bs=12) == UNSUPPORTED
    assert rotate(lib, T=0) == 0
    assert rotate(lib, cache=U8) == INVALID                                     # codes need the fp8 call
    assert rotate(lib, scales=(1.0, 1.0)) == INVALID                            # and it needs codes
    assert rotate(lib, scales=(0.0, 1.0), cache=U8) == INVALID
    assert rotate(lib, scales=(1.0, float("inf")), cache=U8) == INVALID
    assert rotate(lib, dict(k_cache=desc((8, 2, 16, 64), U8, data=0x10004)), scales=(1.0, 1.0), cache=U8) == INVALID
    assert rotate(lib, scales=(1.0, 1.0), cache=U8, T=0) == 0


def bounds(lib, change=(), D=128, bs=16, dt=BF, size=None):
    a = dict(key_bounds=desc((8, 2, 2, D), dt), k_cache=desc((8, 2, bs, D), dt), bt=desc((3, 4), I32), cl=desc((3,), I32),
             qsl=None)
    a.update(change)
    return lib.wllm_update_key_bounds(*refs(a, ("key_bounds", "k_cache", "bt", "cl", "qsl")), size or bs, None)


def test_bounds_refuses(lib):
    assert bounds(lib, dict(key_bounds=desc((8, 2, 2, 128), F16))) == INVALID
    assert bounds(lib, dict(key_bounds=desc((7, 2, 2, 128), BF))) == INVALID
    assert bounds(lib, dict(key_bounds=desc((8, 2, 1, 128), BF))) == INVALID
    assert bounds(lib, dict(key_bounds=desc((8, 2, 2, 128), BF, data=0x10008))) == INVALID
    assert bounds(lib, dict(key_bounds=desc((8, 2, 2, 128), BF, stride=(1024, 512, 256, 1)))) == INVALID
    assert bounds(lib, dict(qsl=desc((3,), I32))) == INVALID                    # B entries, not B + 1
    assert bounds(lib, dict(qsl=desc((4,), I64))) == INVALID
    assert bounds(lib, dict(qsl=desc((4,), I32, stride=(2,)))) == INVALID
    assert bounds(lib, dict(bt=desc((2, 4), I32))) == INVALID
    assert bounds(lib, dict(cl=desc((3,), I64))) == INVALID
    assert bounds(lib, dt=I32) == INVALID
    assert bounds(lib, size=32) == INVALID
    assert bounds(lib, D=96) == UNSUPPORTED
    assert bounds(lib, bs=4) == UNSUPPORTED
    assert bounds(lib, dict(bt=desc((0, 4), I32), cl=desc((0,), I32))) == 0


def select(lib, change=(), B=3, Hq=4, Hkv=2, D=128, bs=16, dt=BF, top=8, sink=1, recent=2, heads=None, mb=40):
    a = dict(sel=desc((B, Hkv, top), I32), q=desc((B, Hq, D), dt), kb=desc((50, Hkv, 2, D), dt), bt=desc((B, mb), I32),
             cl=desc((B,), I32))
    a.update(change)
    return lib.wllm_select_blocks(*refs(a, ("sel", "q", "kb", "bt", "cl")), heads or Hkv, bs, sink, recent, None)


def test_select_refuses(lib):
    assert select(lib, dict(sel=desc((3, 2, 8), I64))) == INVALID
    assert select(lib, dict(sel=desc((3, 4, 8), I32))) == INVALID
    assert select(lib, dict(sel=desc((3, 2, 8), I32, stride=(32, 16, 2)))) == INVALID
    assert select(lib, dict(kb=desc((50, 2, 2, 128), F16))) == INVALID
    assert select(lib, dict(kb=desc((50, 2, 2, 128), U8)), dt=F32) == INVALID
    assert select(lib, dict(kb=desc((50, 2, 128), BF))) == INVALID
    assert select(lib, dict(kb=desc((50, 2, 2, 64), BF))) == INVALID
    assert select(lib, dict(kb=desc((50, 2, 2, 128), BF, data=0x10008))) == INVALID
    assert select(lib, dict(q=desc((3, 4, 128), I32))) == INVALID
    assert select(lib, dict(q=desc((3, 4, 128), BF, stride=(1024, 256, 2)))) == INVALID
    assert select(lib, heads=3) == INVALID
    assert select(lib, Hq=5) == INVALID
    assert select(lib, sink=-1) == INVALID
    assert select(lib, recent=0) == INVALID
    assert select(lib, sink=7, recent=2) == INVALID
    assert select(lib, D=96) == UNSUPPORTED
    assert select(lib, bs=24) == UNSUPPORTED
    assert select(lib, bs=8, mb=200_000) == UNSUPPORTED
    assert select(lib, B=0) == 0
    # a pool without blocks has nothing that a table entry could be clamped to, with query heads or without
    for heads in (4, 0):
        assert select(lib, dict(kb=desc((0, 2, 2, 128), BF, data=None)), Hq=heads) == INVALID


def sparse(lib, change=(), B=3, Hq=4, Hkv=2, D=128, bs=16, dt=BF, cache=None, scale=0.1, scales=None, heads=None, size=None):
    c = cache or dt
    a = dict(out=desc((B, Hq, D), dt), q=desc((B, Hq, D), dt), kc=desc((50, Hkv, bs, D), c), vc=desc((50, Hkv, bs, D), c),
             bt=desc((B, 40), I32), cl=desc((B,), I32), sel=desc((B, Hkv, 8), I32))
    a.update(change)
    args = refs(a, ("out", "q", "kc", "vc", "bt", "cl", "sel"))
    if scales is None:
        return lib.wllm_paged_attention_decode_sparse(*args, heads or Hkv, scale, size or bs, None)
    return lib.wllm_paged_attention_decode_sparse_fp8(*args, heads or Hkv, scale, *scales, size or bs, None)


def test_sparse_refuses(lib):
    assert sparse(lib, dict(sel=desc((3, 2, 8), I64))) == INVALID
    assert sparse(lib, dict(sel=desc((3, 1, 8), I32))) == INVALID
    assert sparse(lib, dict(sel=desc((3, 2, 8), I32, stride=(32, 16, 2)))) == INVALID
    assert sparse(lib, dict(out=desc((3, 4, 128), F16))) == INVALID
    assert sparse(lib, dict(kc=desc((50, 2, 16, 128), F16))) == INVALID
    assert sparse(lib, dict(kc=desc((50, 2, 16, 128), BF, data=0x10008))) == INVALID
    assert sparse(lib, dict(vc=desc((40, 2, 16, 128), BF))) == INVALID
    assert sparse(lib, dict(bt=desc((3, 40), I64))) == INVALID
    assert sparse(lib, dict(cl=desc((2,), I32))) == INVALID
    assert sparse(lib, dict(q=desc((3, 4, 128), BF, data=0x10001), out=desc((3, 4, 128), BF))) == INVALID
    assert sparse(lib, scale=float("nan")) == INVALID
    assert sparse(lib, heads=3) == INVALID
    assert sparse(lib, size=32) == INVALID
    assert sparse(lib, Hq=5) == INVALID
    assert sparse(lib, D=96) == UNSUPPORTED
    assert sparse(lib, bs=4) == UNSUPPORTED
    assert sparse(lib, D=64, bs=8, cache=U8, scales=(1.0, 1.0)) == UNSUPPORTED
    assert sparse(lib, cache=U8) == INVALID
    assert sparse(lib, scales=(1.0, 1.0)) == INVALID
    assert sparse(lib, scales=(1.0, -1.0), cache=U8) == INVALID
    assert sparse(lib, scales=(1.0, 1.0), cache=U8, dt=F32) == INVALID
    assert sparse(lib, B=0) == 0
    assert sparse(lib, scales=(1.0, 1.0), cache=U8, B=0) == 0


@pytest.mark.parametrize("call,name,good", [
    (rotate, "slots", ((6,), I64)), (rotate, "positions", ((6,), I32)), (rotate, "cos_sin", ((100, 64), F32)),
    (rotate, "key", ((6, 2, 64), BF)), (rotate, "q_weight", ((64,), BF)),
    (bounds, "bt", ((3, 4), I32)), (bounds, "cl", ((3,), I32)), (bounds, "qsl", ((4,), I32)),
    (select, "sel", ((3, 2, 8), I32)), (select, "bt", ((3, 40), I32)), (select, "cl", ((3,), I32)), (select, "q", ((3, 4, 128), BF)),
    (sparse, "sel", ((3, 2, 8), I32)), (sparse, "bt", ((3, 40), I32)), (sparse, "cl", ((3,), I32)), (sparse, "out", ((3, 4, 128), BF))])
def test_data_off_its_elements_alignment_is_refused(lib, call, name, good):
    """Half an element off: the kernel's load would be misaligned.  (Nothing is launched: the check comes first.)"""
    n = lib.wllm_launch_count()
    size = torch.empty(0, dtype=good[1]).element_size()
    assert call(lib, {name: desc(*good, data=0x10000 + size // 2)}) == INVALID
    assert b"align" in lib.wllm_last_error() and lib.wllm_launch_count() == n


def test_indices_off_their_alignment_are_refused_by_the_dense_calls(lib):
    x, c = desc((3, 2, 64), BF), desc((8, 2, 16, 64), BF)
    odd = {d: 0x10000 + d // 2 for d in (4, 8)}
    assert lib.wllm_reshape_and_cache(*map(ctypes.byref, (x, x, c, c, desc((3,), I64, data=odd[8]))), None) == INVALID
    assert b"slot_mapping" in lib.wllm_last_error()
    good = dict(bt=desc((3, 4), I32), cl=desc((3,), I32))
    for name, bad in (("bt", desc((3, 4), I32, data=odd[4])), ("cl", desc((3,), I32, data=odd[4]))):
        t = dict(good, **{name: bad})
        assert lib.wllm_paged_attention_decode(*map(ctypes.byref, (x, x, c, c, t["bt"], t["cl"])), 2, 0.1, 16, None) == INVALID
        assert b"align" in lib.wllm_last_error()


def test_binding_refuses():
    x = torch.zeros(2, 2, 64, dtype=BF)
    c = torch.zeros(3, 2, 16, 64, dtype=BF)
    i = torch.zeros(2, dtype=I32)
    with pytest.raises(ValueError, match="CUDA"):
        wllm.rotate_and_cache(x, x, x, x, c, c, i, i, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="style"):
        wllm.rotate_and_cache(x, x, x, x, c, c, i, i, torch.zeros(4, 64), style="thirds")
    with pytest.raises(ValueError, match="sections"):
        wllm.rotate_and_cache(x, x, x, x, c, c, i, i, torch.zeros(4, 64), sections=[16, 16])
    with pytest.raises(ValueError, match="sections"):
        wllm.rotate_and_cache(x, x, x, x, c, c, i, i.view(2, 1), torch.zeros(4, 64))
    with pytest.raises(ValueError, match="at most 4"):
        wllm.rotate_and_cache(x, x, x, x, c, c, i, i.view(2, 1), torch.zeros(4, 64), sections=[8, 8, 8, 4, 4])
    with pytest.raises(ValueError, match="CUDA"):
        wllm.update_key_bounds(c, c, i[:, None], i, 16)
    with pytest.raises(ValueError, match="CUDA"):
        wllm.select_blocks(i, x, c, i, i, 2, 16)
    with pytest.raises(ValueError, match="CUDA"):
        wllm.paged_attention_decode_sparse(x, x, c, c, i, i, i, 2, 0.1, 16)
