"""Inputs and comparisons of the rotary append and block-sparse decode tests (host tensors, seeded)."""
import torch

import oracle

U32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step, relative
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the least value


def bits(x):
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def codes(g, *shape, scale=40.0):
    """E4M3 codes of normal values."""
    return oracle.e4m3_encode(torch.randn(*shape, generator=g) * scale)


def rotary_table(positions, rot, base=1e4):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def block_tables(g, lens, bs, spare=3, width=None):
    """Tables of a shuffled pool, -1 past each sequence's last block, and the pool's number of blocks."""
    counts = [-(-n // bs) for n in lens]
    pool = sum(counts) + spare
    order = torch.randperm(pool, generator=g).to(torch.int32)
    bt = torch.full((len(lens), max(counts + [1]) if width is None else width), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        bt[b, :c] = order[at:at + c]
        at += c
    return bt, pool


def cache(g, pool, hkv, bs, d, dtype, bt=None, lens=None):
    """A pool of normal keys or values; where lengths are given, NaN in every slot that no sequence has."""
    x = codes(g, pool, hkv, bs, d) if dtype == torch.uint8 else randn(g, pool, hkv, bs, d, dtype=dtype)
    if lens is not None:
        live = torch.zeros(pool, bs, dtype=torch.bool)
        for b, n in enumerate(lens):
            for t in range(n):
                live[bt[b, t // bs], t % bs] = True
        nan = torch.tensor(0x7f, dtype=torch.uint8) if dtype == torch.uint8 else torch.tensor(float("nan"), dtype=dtype)
        x = torch.where(live[:, None, :, None], x, nan)
    return x


def assert_turned(got, ref, size, dtype, what):
    """Rows of rotate_and_cache against binary64.  The one rounding to `dtype` is off by at most half a step of the
    result; before it, binary32 operations on a pair of length `size`: the sum of up to 256 squares (16 in a lane's
    chain of fused products, 4 sums across lanes: 20 roundings, halved by the root), the product with 1/D, eps, the
    reciprocal root (2 ulp), two products with it and the weight, two products and a sum of the turn, each at most
    2^-24 relative of `size` or twice that: 32 of them cover it."""
    tol = HALF[dtype] * ref.abs() + 32 * U32 * (1 + HALF[dtype]) * size + TINY[dtype]
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {((got.double() - ref).abs() - tol).max().item():.3g} over"


def assert_codes(got, ref, size, what):
    """E4M3 codes of `ref` (already divided by the scale): half a step is 2^-4 of the value, or 2^-10 (half of the
    least code); binary32 errors as above and one more product."""
    v, r = oracle.widen_e4m3(got), ref.clamp(-448, 448)
    tol = 2.0 ** -4 * r.abs() + 2.0 ** -10 + 36 * U32 * size
    bad = (v - r).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off"


def assert_sparse(got, ref, mag, size, dtype, fp8, what):
    """Attention against binary64.  A weight is off by a factor 1 + d: rounding it to 16 bits (half a step; not for
    f32), the exponential (2^-22 relative, its argument's roundings included as below), and the score's error e^ds - 1
    with ds = size * (rounding of the query to f16 for fp8 caches: 2^-11; binary32 sums of up to 256 products in any
    order: 260 * 2^-24; scaling and difference to the maximum: 6 * 2^-24).  The sum uses the rounded weights, so the
    output moves by at most 2 d sum p |v|; binary32 sums of p v over the tokens and the rescalings stay within
    another 2^-14 of sum p |v| (each rounding 2^-24, 512 of them at most in a chain); and the result is rounded once."""
    ds = size * ((2.0 ** -11 if fp8 and dtype == torch.bfloat16 else 0.0) + 266 * U32)
    d = (HALF[dtype] if dtype != torch.float32 else 0.0) + 2.0 ** -21 + torch.expm1(ds)[..., None]
    tol = (2 * d + 2.0 ** -14 * (0.25 if dtype == torch.float32 else 1.0)) * mag + HALF[dtype] * ref.abs() + 1e-7
    off = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    assert not (off > tol).any(), f"{what}: {int((off > tol).sum())} off, worst {off.max().item():.3g} ({(off / tol).max().item():.2f} of its bound)"
