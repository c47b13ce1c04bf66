"""What the binding offers without a GPU and without its compiled module: the library itself, the host-only calls and
descriptors for callers of the C ABI."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from paged_kv_cache_185_gb300 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def without_module(code):
    """Run code in a process whose import of the compiled module fails."""
    block = "import sys\nsys.modules['paged_kv_cache_185_gb300._describe'] = None\n"
    return subprocess.run([sys.executable, "-c", block + code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_library_and_block_manager_need_no_compiled_module():
    r = without_module("""
import paged_kv_cache_185_gb300 as w
assert "sm_103a" in w.version() and w.launch_count() == 0
m = w.BlockManager(8, 4)
slots, cached = m.add_sequence(1, [1, 2, 3, 4, 5])
assert slots.numel() == 5 and cached == 0 and m.num_free_blocks() == 6
m.close()
lib = w.load_library()
assert lib.wllm_reshape_and_cache(None, None, None, None, None, None) == 1 and b"null" in lib.wllm_last_error()
""")
    assert r.returncode == 0, r.stderr[-1500:]


def test_calls_with_tensors_say_that_the_module_is_missing():
    r = without_module("""
import torch, paged_kv_cache_185_gb300 as w
x, i = torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int64)
for _ in range(2):
    try:
        w.reshape_and_cache(x, x, torch.zeros(3, 2, 16, 64), torch.zeros(3, 2, 16, 64), i)
    except ImportError as e:
        assert "_describe" in str(e)
    else:
        raise AssertionError("no error")
""")
    assert r.returncode == 0, r.stderr[-1500:]


def test_sections_that_do_not_fit_the_struct_are_refused():
    """2^32 + 16 pairs are not 16."""
    x, c = torch.zeros(2, 2, 64), torch.zeros(3, 2, 16, 64)
    i = torch.zeros(2, dtype=torch.int64)
    for n in (2 ** 32 + 16, -2 ** 32 + 16):
        with pytest.raises(ValueError, match="out of range"):
            binding.rotate_and_cache(x, x, x, x, c, c, i, torch.zeros(2, 2, dtype=torch.int64), torch.zeros(4, 64),
                                     sections=[n, 16])


def test_describe_fills_a_descriptor():
    x = torch.zeros(3, 8, 5, dtype=torch.bfloat16)[:, 2:6, ::2]
    d = binding.describe(x)
    assert isinstance(d, binding.WllmTensor) and d.data == x.data_ptr() and (d.dtype, d.ndim) == (2, 3)
    assert list(d.shape) == [3, 4, 3, 0] and list(d.stride) == [40, 5, 2, 0]
    codes = {torch.float32: 0, torch.float16: 1, torch.int32: 3, torch.int64: 4, torch.float8_e4m3fn: 5, torch.uint8: 5}
    for dtype, code in codes.items():
        d = binding.describe(torch.empty(0, 7, dtype=dtype))
        assert d.data is None and d.dtype == code and list(d.shape)[:2] == [0, 7]
    with pytest.raises(ValueError, match="4 dims"):
        binding.describe(torch.zeros(1, 1, 1, 1, 1))
    with pytest.raises(KeyError):
        binding.describe(torch.zeros(1, dtype=torch.float64))
    # as an argument of the C ABI: the call gets as far as the first check that these host tensors fail
    lib = binding.load_library()
    x, c, s = torch.zeros(2, 2, 64), torch.zeros(3, 2, 16, 64), torch.zeros(3, dtype=torch.int64)
    args = [binding.describe(t) for t in (x, x, c, c, s)]
    assert lib.wllm_reshape_and_cache(*map(ctypes.byref, args), None) == binding.WLLM_ERR_INVALID_ARG
    assert b"slot_mapping" in lib.wllm_last_error()
