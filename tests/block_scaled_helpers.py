"""Inputs and comparisons of the tests of the cache with a scale for each block and head (host tensors, seeded)."""
import torch

import oracle
from tests import sparse_helpers as H

U32 = 2.0 ** -24
NAN_CODE = 0x7f


def pool(g, pool_blocks, hkv, bs, d, bt, lens, spread=0.5):
    """Codes and power-of-two scales of a cache; NaN in every slot that no sequence has and in the scales of blocks that
    none names.  `spread`: how far the scales' exponents are apart, as a standard deviation."""
    codes = H.codes(g, pool_blocks, hkv, bs, d, scale=100.0)
    e = (torch.randn(pool_blocks, hkv, generator=g) * spread - 6).round().clamp(-40, 40)
    scales = torch.exp2(e).float()
    live = torch.zeros(pool_blocks, bs, dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            live[bt[b, t // bs], t % bs] = True
    codes = torch.where(live[:, None, :, None], codes, torch.tensor(NAN_CODE, dtype=torch.uint8))
    scales = torch.where(live.any(1)[:, None], scales, torch.tensor(float("nan")))
    return codes, scales


def assert_attention(got, ref, mag, size, least, dtype, what):
    """Attention against binary64.  A weight's relative error d: its rounding to f16, at most half a step, 2^-11, while
    it is a normal number; the exponential, 2^-21 with its argument's subtraction; and the score's error e^ds - 1 with
    ds = size * (binary32 sums of up to 256 products in any order, scaling by the query's and the block's factors, the
    query's rounding: 270 * 2^-24) + the logarithm of the value's scale and the sum with it (2^-21 and 40 * 2^-23).  The
    sum l takes the weights unrounded.  So the output moves by at most (2 d) sum p |v|, and another 2^-14 of it for the
    binary32 sums.  Weights below 2^-14 of f16 are off by at most 2^-25, the largest one being 2^7 at least: with codes
    up to 448 that is 448 * 2^-32 of a token's value scale each.  The result is rounded once."""
    ds = size * 270 * U32 + 2.0 ** -21 + 40 * 2.0 ** -23
    d = 2.0 ** -11 + 2.0 ** -21 + torch.expm1(ds)[..., None]
    tol = (2 * d + 2.0 ** -14) * mag + 448 * 2.0 ** -32 * least[..., None] + H.HALF[dtype] * ref.abs() + H.TINY[dtype]
    off = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    assert not (off > tol).any(), f"{what}: {int((off > tol).sum())} off, worst {off.max().item():.3g} ({(off / tol).max().item():.2f} of its bound)"


def same_codes(got, ref, what):
    """Codes equal bit for bit, NaN with NaN."""
    a, b = oracle.widen_e4m3(got), oracle.widen_e4m3(ref)
    same = (got == ref) | (a.isnan() & b.isnan())
    assert same.all(), f"{what}: {int((~same).sum())} codes differ, first at {torch.nonzero(~same)[0].tolist()}"
