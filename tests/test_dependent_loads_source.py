"""Kernels launched as programmatic dependents are alive while the kernel before them writes their inputs.  A non-coherent
load is defined only for memory that nobody writes during the kernel's life, so their sources use none."""
import os
import re

import pytest

from paged_kv_cache_185_gb300 import build


@pytest.mark.parametrize("name", ["rotate_kernel.cuh", "key_bounds.cu", "select.cu", "sparse_decode.cu"])
def test_dependent_kernels_use_plain_loads(name):
    text = open(os.path.join(build.CSRC, name)).read()
    code = re.sub(r"//.*", "", text)
    assert "launch_dependent(" in code and "grid_wait()" in code
    assert not re.search(r"__ldg|__ldcs|ld\.global\.nc|\b__restrict__", code)
