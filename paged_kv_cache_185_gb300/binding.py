"""ctypes binding over libwllm.so (C ABI in include/wllm.h).

Argument marshalling only: each call turns torch tensors into ``wllm_tensor``
descriptors (device pointer, dtype code, sizes, strides in elements), passes
the current CUDA stream (the compiled module ``_describe`` does both), and
raises ``WllmError`` on a non-zero status.  Every
step of the computation runs in the library's CUDA kernels; there is no CPU
path.  Loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libwllm.so")

WLLM_OK, WLLM_ERR_INVALID_ARG, WLLM_ERR_UNSUPPORTED, WLLM_ERR_OUT_OF_RANGE, WLLM_ERR_CUDA = range(5)
# E4M3 caches may be passed as torch.float8_e4m3fn or as raw uint8 codes
_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int32: 3, torch.int64: 4,
          torch.float8_e4m3fn: 5, torch.uint8: 5}

# every symbol include/wllm.h declares
EXPORTED = ("wllm_reshape_and_cache", "wllm_paged_attention_decode", "wllm_decode_step",
            "wllm_reshape_and_cache_fp8", "wllm_paged_attention_decode_fp8", "wllm_decode_step_fp8",
            "wllm_paged_attention_prefill", "wllm_paged_attention_prefill_fp8",
            "wllm_paged_attention_decode_noalloc",
            "wllm_rotate_and_cache", "wllm_rotate_and_cache_fp8", "wllm_update_key_bounds", "wllm_select_blocks",
            "wllm_paged_attention_decode_sparse", "wllm_paged_attention_decode_sparse_fp8",
            "wllm_paged_attention_workspace_bytes", "wllm_set_workspace",
            "wllm_partition_tokens", "wllm_device_errors", "wllm_selftest_wait_timeout", "wllm_launch_count",
            "wllm_last_error", "wllm_version",
            "wllm_bm_create", "wllm_bm_destroy", "wllm_bm_add_sequence", "wllm_bm_append_token",
            "wllm_bm_fork", "wllm_bm_free_sequence", "wllm_bm_block_table", "wllm_bm_num_free_blocks",
            "wllm_bm_num_cached_blocks", "wllm_bm_block_ref")


class WllmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"wllm status {status}: {message}")
        self.status = status


class WllmTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class WllmRotary(ctypes.Structure):
    _fields_ = [("style", ctypes.c_int32), ("num_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4),
                ("eps", ctypes.c_float)]


_ROTARY_STYLE = {"halves": 0, "adjacent": 1}


_lib = None
_entries = {}   # entry points that take tensors first: name -> what _invoke takes
_invoke = None  # _describe.call, from the first call with tensors on
_lock = threading.Lock()


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libwllm.so (raises if it is missing: build it with ``build()`` first)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: run `python -m paged_kv_cache_185_gb300.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        P = ctypes.POINTER(WllmTensor)
        lib.wllm_reshape_and_cache.argtypes = [P, P, P, P, P, ctypes.c_void_p]
        lib.wllm_reshape_and_cache.restype = ctypes.c_int
        lib.wllm_paged_attention_decode.argtypes = [P, P, P, P, P, P, ctypes.c_int, ctypes.c_float,
                                                    ctypes.c_int, ctypes.c_void_p]
        lib.wllm_paged_attention_decode.restype = ctypes.c_int
        lib.wllm_decode_step.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_int, ctypes.c_float, ctypes.c_int,
                                         ctypes.c_void_p]
        lib.wllm_decode_step.restype = ctypes.c_int
        f32 = ctypes.c_float
        lib.wllm_reshape_and_cache_fp8.argtypes = [P, P, P, P, P, f32, f32, ctypes.c_void_p]
        lib.wllm_reshape_and_cache_fp8.restype = ctypes.c_int
        lib.wllm_paged_attention_decode_fp8.argtypes = [P, P, P, P, P, P, ctypes.c_int, f32, f32, f32,
                                                        ctypes.c_int, ctypes.c_void_p]
        lib.wllm_paged_attention_decode_fp8.restype = ctypes.c_int
        lib.wllm_decode_step_fp8.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_int, f32, f32, f32, ctypes.c_int,
                                             ctypes.c_void_p]
        lib.wllm_decode_step_fp8.restype = ctypes.c_int
        lib.wllm_paged_attention_prefill.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, ctypes.c_float,
                                                     ctypes.c_int, ctypes.c_void_p]
        lib.wllm_paged_attention_prefill.restype = ctypes.c_int
        lib.wllm_paged_attention_prefill_fp8.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, f32, f32, f32,
                                                         ctypes.c_int, ctypes.c_void_p]
        lib.wllm_paged_attention_prefill_fp8.restype = ctypes.c_int
        lib.wllm_paged_attention_decode_noalloc.argtypes = [P, P, P, P, P, P, ctypes.c_int, ctypes.c_float,
                                                            ctypes.c_int, ctypes.c_void_p]
        lib.wllm_paged_attention_decode_noalloc.restype = ctypes.c_int
        how = ctypes.POINTER(WllmRotary)
        lib.wllm_rotate_and_cache.argtypes = [P] * 11 + [how, ctypes.c_void_p]
        lib.wllm_rotate_and_cache.restype = ctypes.c_int
        lib.wllm_rotate_and_cache_fp8.argtypes = [P] * 11 + [how, f32, f32, ctypes.c_void_p]
        lib.wllm_rotate_and_cache_fp8.restype = ctypes.c_int
        lib.wllm_update_key_bounds.argtypes = [P] * 5 + [ctypes.c_int, ctypes.c_void_p]
        lib.wllm_update_key_bounds.restype = ctypes.c_int
        lib.wllm_select_blocks.argtypes = [P] * 5 + [ctypes.c_int] * 4 + [ctypes.c_void_p]
        lib.wllm_select_blocks.restype = ctypes.c_int
        lib.wllm_paged_attention_decode_sparse.argtypes = [P] * 7 + [ctypes.c_int, f32, ctypes.c_int, ctypes.c_void_p]
        lib.wllm_paged_attention_decode_sparse.restype = ctypes.c_int
        lib.wllm_paged_attention_decode_sparse_fp8.argtypes = [P] * 7 + [ctypes.c_int, f32, f32, f32, ctypes.c_int,
                                                                       ctypes.c_void_p]
        lib.wllm_paged_attention_decode_sparse_fp8.restype = ctypes.c_int
        lib.wllm_paged_attention_workspace_bytes.argtypes = [ctypes.c_int] * 6
        lib.wllm_paged_attention_workspace_bytes.restype = ctypes.c_size_t
        lib.wllm_set_workspace.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
        lib.wllm_set_workspace.restype = ctypes.c_int
        lib.wllm_partition_tokens.argtypes = [ctypes.c_int] * 7
        lib.wllm_partition_tokens.restype = ctypes.c_int
        lib.wllm_device_errors.argtypes = []
        lib.wllm_device_errors.restype = ctypes.c_int
        lib.wllm_selftest_wait_timeout.argtypes = [ctypes.c_ulonglong, ctypes.c_void_p]
        lib.wllm_selftest_wait_timeout.restype = ctypes.c_int
        lib.wllm_launch_count.argtypes = []
        lib.wllm_launch_count.restype = ctypes.c_ulonglong
        lib.wllm_last_error.argtypes = []
        lib.wllm_last_error.restype = ctypes.c_char_p
        lib.wllm_version.argtypes = []
        lib.wllm_version.restype = ctypes.c_char_p
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        p64, p32 = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int32)
        lib.wllm_bm_create.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp)]
        lib.wllm_bm_create.restype = ctypes.c_int
        lib.wllm_bm_destroy.argtypes = [vp]
        lib.wllm_bm_destroy.restype = None
        lib.wllm_bm_add_sequence.argtypes = [vp, i64, p32, i64, p64, p64]
        lib.wllm_bm_add_sequence.restype = ctypes.c_int
        lib.wllm_bm_append_token.argtypes = [vp, i64, i32, p64, p32, p32]
        lib.wllm_bm_append_token.restype = ctypes.c_int
        lib.wllm_bm_fork.argtypes = [vp, i64, i64]
        lib.wllm_bm_fork.restype = ctypes.c_int
        lib.wllm_bm_free_sequence.argtypes = [vp, i64]
        lib.wllm_bm_free_sequence.restype = ctypes.c_int
        lib.wllm_bm_block_table.argtypes = [vp, i64, p32, ctypes.c_int, p64]
        lib.wllm_bm_block_table.restype = ctypes.c_int
        lib.wllm_bm_num_free_blocks.argtypes = [vp]
        lib.wllm_bm_num_free_blocks.restype = i64
        lib.wllm_bm_num_cached_blocks.argtypes = [vp]
        lib.wllm_bm_num_cached_blocks.restype = i64
        lib.wllm_bm_block_ref.argtypes = [vp, i32]
        lib.wllm_bm_block_ref.restype = ctypes.c_int
        _lib = lib
    return _lib


def _load_calls():
    """Bind the entry points that take tensors through the compiled module, which needs torch's libraries; the library
    itself and its host-only calls do not."""
    global _invoke
    lib = load_library()
    with _lock:
        if _invoke is not None:
            return
        from . import build
        if build.described_for() not in ("", build.describe_key()):
            raise ImportError(f"_describe.so was built for {build.described_for()!r}, this process has "
                              f"{build.describe_key()!r}: run `python -m paged_kv_cache_185_gb300.build`")
        from . import _describe as module
        for name in EXPORTED:
            f = getattr(lib, name)
            if f.argtypes and f.argtypes[0] is ctypes.POINTER(WllmTensor):
                _entries[name] = module.bind(name, ctypes.cast(f, ctypes.c_void_p).value)
        _invoke = module.call


def describe(t: torch.Tensor) -> WllmTensor:
    """The descriptor of a tensor, for callers of the C ABI through ctypes (the tensor has to outlive its use)."""
    if t.dim() > 4:
        raise ValueError("at most 4 dims")
    d = WllmTensor(t.data_ptr() if t.numel() > 0 else None, _DTYPE[t.dtype], t.dim())
    d.shape[:t.dim()] = t.shape
    d.stride[:t.dim()] = t.stride()
    return d


def _stream_handle(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _check(rc: int) -> None:
    if rc != WLLM_OK:
        raise WllmError(rc, load_library().wllm_last_error().decode())


def _call(name: str, tensors, *scalars) -> None:
    """Entry point ``name`` on ``tensors`` (None: not given) and ``scalars``, on the current stream of the tensors'
    device.  Host tensors, or tensors of several devices, raise ValueError."""
    if _invoke is None:
        _load_calls()
    rc = _invoke(_entries[name], tensors, *scalars)
    if rc != WLLM_OK:
        _check(rc)


def reshape_and_cache(key, value, k_cache, v_cache, slot_mapping) -> None:
    """KV append: scatter key/value [T,Hkv,D] into caches [N_b,Hkv,bs,D] at ``slot_mapping``."""
    _call("wllm_reshape_and_cache", (key, value, k_cache, v_cache, slot_mapping))


def paged_attention_decode(out, q, k_cache, v_cache, block_tables, context_lens,
                           num_kv_heads: int, scale: float, block_size: int) -> torch.Tensor:
    """Paged decode attention into ``out`` [B,Hq,D]; returns ``out``."""
    _call("wllm_paged_attention_decode", (out, q, k_cache, v_cache, block_tables, context_lens),
          int(num_kv_heads), float(scale), int(block_size))
    return out


def paged_attention_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens,
                                   num_kv_heads: int, scale: float, block_size: int) -> torch.Tensor:
    """Paged decode attention that allocates no device memory (fixed scratch
    inside the library; see wllm_paged_attention_decode_noalloc in wllm.h)."""
    _call("wllm_paged_attention_decode_noalloc", (out, q, k_cache, v_cache, block_tables, context_lens),
          int(num_kv_heads), float(scale), int(block_size))
    return out


def decode_step(out, q, key, value, k_cache, v_cache, slot_mapping, block_tables, context_lens,
                num_kv_heads: int, scale: float, block_size: int) -> torch.Tensor:
    """One decode step of one layer: append this step's K/V, then attend (one
    fused launch where the kernel allows; see wllm_decode_step)."""
    _call("wllm_decode_step", (out, q, key, value, k_cache, v_cache, slot_mapping, block_tables, context_lens),
          int(num_kv_heads), float(scale), int(block_size))
    return out


def reshape_and_cache_fp8(key, value, k_cache, v_cache, slot_mapping, k_scale: float, v_scale: float) -> None:
    """KV append into E4M3 caches (uint8 or float8_e4m3fn): stores E4M3(x * (1/scale))."""
    _call("wllm_reshape_and_cache_fp8", (key, value, k_cache, v_cache, slot_mapping), float(k_scale), float(v_scale))


def paged_attention_decode_fp8(out, q, k_cache, v_cache, block_tables, context_lens, num_kv_heads: int,
                               scale: float, k_scale: float, v_scale: float, block_size: int) -> torch.Tensor:
    """Paged decode attention over E4M3 caches (K = code * k_scale, V = code * v_scale); returns ``out``."""
    _call("wllm_paged_attention_decode_fp8", (out, q, k_cache, v_cache, block_tables, context_lens),
          int(num_kv_heads), float(scale), float(k_scale), float(v_scale), int(block_size))
    return out


def decode_step_fp8(out, q, key, value, k_cache, v_cache, slot_mapping, block_tables, context_lens,
                    num_kv_heads: int, scale: float, k_scale: float, v_scale: float, block_size: int) -> torch.Tensor:
    """decode_step over E4M3 caches: the append quantises with the same scales the attention reads back."""
    _call("wllm_decode_step_fp8", (out, q, key, value, k_cache, v_cache, slot_mapping, block_tables, context_lens),
          int(num_kv_heads), float(scale), float(k_scale), float(v_scale), int(block_size))
    return out


def paged_attention_prefill(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                            num_kv_heads: int, scale: float, block_size: int) -> torch.Tensor:
    """Chunked-prefill paged attention into ``out`` [T,Hq,D] (packed chunks, causal); returns ``out``."""
    _call("wllm_paged_attention_prefill", (out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc),
          int(num_kv_heads), float(scale), int(block_size))
    return out


def paged_attention_prefill_fp8(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                                num_kv_heads: int, scale: float, k_scale: float, v_scale: float,
                                block_size: int) -> torch.Tensor:
    """Chunked-prefill paged attention over E4M3 caches (K = code * k_scale, V = code * v_scale)."""
    _call("wllm_paged_attention_prefill_fp8", (out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc),
          int(num_kv_heads), float(scale), float(k_scale), float(v_scale), int(block_size))
    return out


@functools.lru_cache(maxsize=256)
def _rotary(style, sections, eps):
    """The options of a rotary call as a C struct, which is never written again, and its address."""
    if style not in _ROTARY_STYLE:
        raise ValueError(f"style must be one of {sorted(_ROTARY_STYLE)}, got {style!r}")
    if len(sections) > 4:
        raise ValueError("at most 4 sections")
    if any(abs(n) > 0x7fffffff for n in sections):
        raise ValueError(f"sections out of range: {sections}")
    how = WllmRotary(_ROTARY_STYLE[style], max(1, len(sections)))
    how.sections[:len(sections)] = sections
    how.eps = eps
    return how, ctypes.addressof(how)


def _rotate(name, tensors, eps, style, sections, scales):
    positions = tensors[7]
    if sections is None:
        sections = ()
        if positions.dim() == 2 and positions.shape[0] > 1:
            raise ValueError("positions on several axes need sections")
    else:
        sections = tuple(int(n) for n in sections)
        if len(sections) > 1 and positions.dim() == 1:
            raise ValueError("several sections need positions [axes, T]")
    how = _rotary(style, sections, float(eps))  # held until the call returns
    _call(name, tensors, how[1], *scales)


def rotate_and_cache(q_out, q, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin, *, q_weight=None,
                     k_weight=None, eps: float = 1e-6, style: str = "halves", sections=None) -> torch.Tensor:
    """Rotary append: per-head norms of q and key (where a weight [D] is given), rotary positions from the table
    ``cos_sin`` [P,R] (cosines, then sines), query into ``q_out`` (may be ``q``), key and value to their slots.

    ``positions`` is [T], or [axes,T] with ``sections`` naming the pairs that each axis turns.  ``style``:
    "halves" pairs elements (i, i+R/2), "adjacent" (2i, 2i+1).  Returns ``q_out``."""
    _rotate("wllm_rotate_and_cache", (q_out, q, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin, q_weight,
                                      k_weight), eps, style, sections, ())
    return q_out


def rotate_and_cache_fp8(q_out, q, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin, k_scale: float,
                         v_scale: float, *, q_weight=None, k_weight=None, eps: float = 1e-6, style: str = "halves",
                         sections=None) -> torch.Tensor:
    """rotate_and_cache into E4M3 caches: stores E4M3(x * (1/scale)) of the turned keys and of the values."""
    _rotate("wllm_rotate_and_cache_fp8", (q_out, q, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin,
                                          q_weight, k_weight), eps, style, sections, (float(k_scale), float(v_scale)))
    return q_out


def update_key_bounds(key_bounds, k_cache, block_tables, context_lens, block_size: int,
                      query_start_loc=None) -> torch.Tensor:
    """Least and greatest key elements, ``key_bounds`` [N_b,Hkv,2,D], of every block that the new tokens filled:
    the last ``query_start_loc[b+1] - query_start_loc[b]`` of each sequence, or one each.  Returns ``key_bounds``."""
    _call("wllm_update_key_bounds", (key_bounds, k_cache, block_tables, context_lens, query_start_loc), int(block_size))
    return key_bounds


def select_blocks(selected, q, key_bounds, block_tables, context_lens, num_kv_heads: int, block_size: int,
                  num_sink: int = 0, num_recent: int = 1) -> torch.Tensor:
    """The blocks that each sequence's query should read, ``selected`` [B,Hkv,top] int32 (ascending, then -1): the
    first ``num_sink``, the last ``num_recent``, and those whose key bounds allow the largest scores."""
    _call("wllm_select_blocks", (selected, q, key_bounds, block_tables, context_lens),
          int(num_kv_heads), int(block_size), int(num_sink), int(num_recent))
    return selected


def paged_attention_decode_sparse(out, q, k_cache, v_cache, block_tables, context_lens, selected, num_kv_heads: int,
                                  scale: float, block_size: int) -> torch.Tensor:
    """Paged decode attention over the blocks listed in ``selected`` [B,Hkv,top] only; returns ``out``."""
    _call("wllm_paged_attention_decode_sparse", (out, q, k_cache, v_cache, block_tables, context_lens, selected),
          int(num_kv_heads), float(scale), int(block_size))
    return out


def paged_attention_decode_sparse_fp8(out, q, k_cache, v_cache, block_tables, context_lens, selected,
                                      num_kv_heads: int, scale: float, k_scale: float, v_scale: float,
                                      block_size: int) -> torch.Tensor:
    """paged_attention_decode_sparse over E4M3 caches (K = code * k_scale, V = code * v_scale); returns ``out``."""
    _call("wllm_paged_attention_decode_sparse_fp8", (out, q, k_cache, v_cache, block_tables, context_lens, selected),
          int(num_kv_heads), float(scale), float(k_scale), float(v_scale), int(block_size))
    return out


def workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size) -> int:
    return int(load_library().wllm_paged_attention_workspace_bytes(
        num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size))


def set_workspace(buf: torch.Tensor | None) -> None:
    """Use a caller-owned device buffer (uint8, 256-byte aligned) as workspace; None reverts."""
    lib = load_library()
    if buf is None:
        _check(lib.wllm_set_workspace(None, 0))
    else:
        with torch.cuda.device(buf.device):
            _check(lib.wllm_set_workspace(buf.data_ptr(), buf.numel() * buf.element_size()))


def partition_tokens(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size,
                     dtype: torch.dtype) -> int:
    return int(load_library().wllm_partition_tokens(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                    max_blocks_per_seq, block_size, _DTYPE[dtype]))


def device_errors() -> int:
    return int(load_library().wllm_device_errors())


def selftest_wait_timeout(limit_ns: int, device=None) -> None:
    """Run the bounded-wait self-test kernel on the current stream (see
    wllm_selftest_wait_timeout); call device_errors() afterwards."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    lib = load_library()
    with torch.cuda.device(dev):
        _check(lib.wllm_selftest_wait_timeout(int(limit_ns), _stream_handle(dev)))


def launch_count() -> int:
    """Kernel launches the library has issued in this process."""
    return int(load_library().wllm_launch_count())


def version() -> str:
    return load_library().wllm_version().decode()


class BlockManager:
    """Prefix-caching manager of the physical KV blocks (host side; see the
    wllm_bm_* calls in wllm.h).  Argument marshalling only."""

    def __init__(self, num_blocks: int, block_size: int):
        self._lib = load_library()
        h = ctypes.c_void_p()
        rc = self._lib.wllm_bm_create(int(num_blocks), int(block_size), ctypes.byref(h))
        if rc != WLLM_OK:
            raise WllmError(rc, "wllm_bm_create")
        self._h = h
        self.num_blocks, self.block_size = int(num_blocks), int(block_size)

    def close(self):
        if self._h:
            self._lib.wllm_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _ok(rc: int, what: str):
        if rc != WLLM_OK:
            raise WllmError(rc, what)

    def add_sequence(self, seq_id: int, tokens):
        """Returns (slots [n] int64 tensor, number of leading tokens already cached)."""
        t = torch.as_tensor(tokens, dtype=torch.int32).contiguous()
        n = t.numel()
        slots = torch.empty(n, dtype=torch.int64)
        cached = ctypes.c_int64()
        self._ok(self._lib.wllm_bm_add_sequence(
            self._h, int(seq_id), ctypes.cast(t.data_ptr(), ctypes.POINTER(ctypes.c_int32)) if n else None, n,
            ctypes.cast(slots.data_ptr(), ctypes.POINTER(ctypes.c_int64)) if n else None, ctypes.byref(cached)),
            "wllm_bm_add_sequence")
        return slots, int(cached.value)

    def append_token(self, seq_id: int, token: int):
        """Returns (slot, copy) with copy = (src_block, dst_block) or None."""
        slot, src, dst = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
        self._ok(self._lib.wllm_bm_append_token(self._h, int(seq_id), int(token), ctypes.byref(slot),
                                                ctypes.byref(src), ctypes.byref(dst)), "wllm_bm_append_token")
        return int(slot.value), (None if src.value < 0 else (int(src.value), int(dst.value)))

    def fork(self, parent: int, child: int):
        self._ok(self._lib.wllm_bm_fork(self._h, int(parent), int(child)), "wllm_bm_fork")

    def free_sequence(self, seq_id: int):
        self._ok(self._lib.wllm_bm_free_sequence(self._h, int(seq_id)), "wllm_bm_free_sequence")

    def block_table(self, seq_id: int, max_blocks: int):
        """Returns (row [max_blocks] int32 tensor, -1 past the last block; context length)."""
        row = torch.empty(int(max_blocks), dtype=torch.int32)
        n = ctypes.c_int64()
        self._ok(self._lib.wllm_bm_block_table(
            self._h, int(seq_id), ctypes.cast(row.data_ptr(), ctypes.POINTER(ctypes.c_int32)) if max_blocks else None,
            int(max_blocks), ctypes.byref(n)), "wllm_bm_block_table")
        return row, int(n.value)

    def num_free_blocks(self) -> int:
        return int(self._lib.wllm_bm_num_free_blocks(self._h))

    def num_cached_blocks(self) -> int:
        return int(self._lib.wllm_bm_num_cached_blocks(self._h))

    def block_ref(self, block: int) -> int:
        return int(self._lib.wllm_bm_block_ref(self._h, int(block)))
