"""What block selection assumes of the tensor cores, measured: two chained mma.sync m16n8k16 from zero are within
136 * 2^-24 of the magnitudes of their 32 products (34 * 2^-22: 22 bits kept of each of 17 terms, twice).  The hardware's
documents promise no such bound; the selection is exact where it holds."""
import ctypes
import os
import subprocess

import pytest
import torch

from paged_kv_cache_185_gb300 import build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
BF, F16 = torch.bfloat16, torch.float16
BOUND = 136 * 2.0 ** -24


@pytest.fixture(scope="module")
def chain(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("mma") / "mma_rounding.so")
    subprocess.run([build._nvcc(), *build.ARCH, "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", build.CSRC,
                    os.path.join(HERE, "mma_rounding.cu"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.mma_chain.argtypes = [ctypes.c_int, ctypes.c_int] + [ctypes.c_void_p] * 3

    def run(a, b):
        n = a.shape[0]
        assert a.shape == (n, 2, 16, 16) and b.shape == (n, 2, 16, 8) and a.dtype == b.dtype
        ad, bd, d = a.contiguous().cuda(), b.contiguous().cuda(), torch.empty(n, 16, 8, device="cuda")
        torch.cuda.synchronize()
        assert lib.mma_chain(int(a.dtype == BF), n, ad.data_ptr(), bd.data_ptr(), d.data_ptr()) == 0
        return d.cpu().double()

    return run


def worst(chain, a, b):
    ref = torch.einsum("nsik,nskj->nij", a.double(), b.double())
    mag = torch.einsum("nsik,nskj->nij", a.double().abs(), b.double().abs())
    off = (chain(a, b) - ref).abs()
    assert (off[mag == 0] == 0).all()
    return (off / mag.clamp(min=1e-300)).max().item()


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("spread", [0, 4, 12, 24])
def test_random_products(chain, dtype, spread):
    """Normal values times powers of two up to 2^spread apart (within f16's normal range)."""
    g = torch.Generator().manual_seed(spread)
    n = 4000
    scale = lambda *s: 2.0 ** torch.randint(-(spread // 2), spread // 2 + 1, s, generator=g).double()  # noqa: E731
    a = (torch.randn(n, 2, 16, 16, generator=g).double() * scale(n, 2, 16, 16)).to(dtype)
    b = (torch.randn(n, 2, 16, 8, generator=g).double() * scale(n, 2, 16, 8) * 2.0 ** -3).to(dtype)
    assert worst(chain, a, b) <= BOUND


@pytest.mark.parametrize("dtype", [BF, F16])
def test_products_that_cancel(chain, dtype):
    """Large products that cancel, in one instruction or across the two, over small ones down to 2^-30 of them."""
    g = torch.Generator().manual_seed(5)
    n = 4000
    a = torch.randn(n, 2, 16, 16, generator=g).to(dtype)
    b = (torch.randn(n, 2, 16, 8, generator=g) * 2.0 ** torch.randint(-14, 1, (n, 2, 16, 1), generator=g).double()).to(dtype)
    for m in range(n):
        i, j = torch.randperm(16, generator=g)[:2].tolist()
        s, t = (0, 0) if m % 3 == 0 else (1, 1) if m % 3 == 1 else (0, 1)
        big = 2.0 ** (m % 9)
        a[m, s, :, i], a[m, t, :, j] = 1.5 * big, -1.5 * big
        b[m, s, i], b[m, t, j] = 1.25 * big, 1.25 * big
    assert worst(chain, a, b) <= BOUND


@pytest.mark.parametrize("dtype", [BF, F16])
def test_each_small_product_beside_a_large_one(chain, dtype):
    """One product of 1 and 31 alike of 2^-k: what is cut off each of them adds up."""
    a = torch.ones(24, 2, 16, 16, dtype=dtype)
    b = torch.zeros(24, 2, 16, 8, dtype=torch.float64)
    for k in range(24):
        b[k] = 2.0 ** -k * (1 + 2.0 ** -7) if k < 15 or dtype == BF else 2.0 ** -14
        b[k, 0, 3] = 1.0
        if k >= 15 and dtype == F16:
            a[k] = 2.0 ** (14 - k)
            a[k, 0, :, 3] = 1.0
    assert worst(chain, a, b.to(dtype)) <= BOUND
