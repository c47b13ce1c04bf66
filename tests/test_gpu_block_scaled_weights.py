"""The softmax weights of the attention over a block-scaled cache reach the output unrounded."""
import pytest
import torch

import paged_kv_cache_185_gb300 as wllm
from oracle import block_scaled as S
from tests import block_scaled_helpers as K
from tests import sparse_helpers as H

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
SCALE = 0.002


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def assert_kept(got, ref, mag, size, d, dtype):
    """Short contexts and small scores, so that everything but the output's own rounding is small.

    The products q.k take head_dim / 16 instructions, each within 17 * 2^-22 of the magnitudes of its 16 products and sum;
    query rows are exact in f16 behind their power of two.  With 8 roundings of factors and sums a score is off by at most
    size * (head_dim / 16 * 17 * 2^-22 + 8 * 2^-24), size = max scale sum |q k|.  To the base 2 it meets the logarithm of the
    value's scale and the shift, below 32 together (asserted): its 2^-22 and 3 roundings of the sum and of the difference to
    the maximum are 32 * (2^-22 + 3 * 2^-24) = 56 * 2^-22, the exponential 2^-22 more.  All this counts twice, in numerator
    and sum.  Two words of f16 leave off 2^-10 * 2^-11 of a weight, or at the subnormal end 2^-25 where the largest is 2^7 at
    least, 2^-32 of n weights: below 2^-20 with weights within 2^4 of one another (asserted).  The products with v are 8
    instructions at most (64 tokens, two words), each within 17 * 2^-22; sums, merging and scaling 40 roundings.  One word
    alone would leave off up to 2^-12 of a weight, several times this bound."""
    assert 2 * size.max() < 4
    ds = size * (d / 16 * 17 * 2.0 ** -22 + 8 * H.U32)
    rel = 2 * (torch.expm1(ds)[..., None] + 57 * 2.0 ** -22) + 2.0 ** -20 + 8 * 17 * 2.0 ** -22 + 40 * H.U32
    tol = rel * mag + H.HALF[dtype] * ref.abs() + H.TINY[dtype]
    off = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all()
    assert (off <= tol).all(), f"{int((off > tol).sum())} of {off.numel()} off, worst {(off / tol).max().item():.2f} of its bound"


def case(seed, dtype, lens, rows, hq, hkv, d, bs):
    g = H.gen(seed)
    bt, blocks = H.block_tables(g, lens, bs)
    (kc, ks), (vc, vs) = (K.pool(g, blocks, hkv, bs, d, bt, lens) for _ in range(2))
    named = vs[~vs.isnan()]
    assert named.max() / named.min() <= 16 and named.log2().abs().max() < 16
    return [H.randn(g, rows, hq, d, dtype=dtype), kc, vc, ks, vs, bt, i32(lens)]


FORMS = [(8, 1, 64, 16), (6, 2, 128, 8), (16, 1, 128, 16), (32, 2, 64, 32), (4, 4, 256, 16)]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("hq,hkv,d,bs", FORMS)
def test_decode_keeps_its_weights(dtype, hq, hkv, d, bs):
    lens = [2 + i % 15 for i in range(45)]
    x = case(hq + d, dtype, lens, 45, hq, hkv, d, bs)
    out = torch.empty_like(x[0]).cuda()
    wllm.paged_attention_decode_block_scaled(out, *(t.cuda() for t in x), hkv, SCALE, bs)
    ref, mag, size, _ = S.attention(*x, SCALE)
    assert_kept(out.cpu(), ref, mag, size, d, dtype)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("hq,hkv,d,bs", [f for f in FORMS if f[2] < 256])
def test_prefill_keeps_its_weights(dtype, hq, hkv, d, bs):
    lens = [2 + i % 15 for i in range(30)]
    new = [min(n, 1 + i % 7) for i, n in enumerate(lens)]
    starts = i32([0] + torch.tensor(new).cumsum(0).tolist())
    x = case(hq + d + 1, dtype, lens, int(starts[-1]), hq, hkv, d, bs)
    out = torch.empty_like(x[0]).cuda()
    wllm.paged_attention_prefill_block_scaled(out, *(t.cuda() for t in x), starts.cuda(), hkv, SCALE, bs)
    ref, mag, size, _ = S.attention(*x, SCALE, starts)
    assert_kept(out.cpu(), ref, mag, size, d, dtype)
