"""NaN codes of a block-scaled cache reach the outputs that see their tokens, and no other."""
import pytest
import torch

import paged_kv_cache_185_gb300 as wllm
from oracle import block_scaled as S
from tests import block_scaled_helpers as K
from tests import sparse_helpers as H

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
BS, D = 16, 128


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def check(dtype, lens, new, hq, hkv, keys, values, decode=False):
    """`keys`: (sequence, token, kv head, element) of keys that become NaN; `values` alike."""
    g = H.gen(len(lens) + sum(lens))
    bt, blocks = H.block_tables(g, lens, BS)
    (kc, ks), (vc, vs) = (K.pool(g, blocks, hkv, BS, D, bt, lens) for _ in range(2))
    starts = i32([0] + torch.tensor(new).cumsum(0).tolist())
    q = H.randn(g, int(starts[-1]), hq, D, dtype=dtype)
    more = () if decode else (starts,)
    ref, mag, size, least = S.attention(q, kc, vc, ks, vs, bt, i32(lens), 0.05, *more)
    bad = torch.zeros(ref.shape, dtype=torch.bool)
    group = hq // hkv
    for kind, cache, at in (("k", kc, keys), ("v", vc, values)):
        for b, t, h, d in at:
            cache[bt[b, t // BS], h, t % BS, d] = K.NAN_CODE
            first = int(starts[b + 1]) - (lens[b] - t)  # the row of token t, if the chunk has it
            rows = slice(max(int(starts[b]), first), int(starts[b + 1]))
            bad[rows, h * group:(h + 1) * group, slice(None) if kind == "k" else d] = True
    assert bad.any() and not bad.all()
    out = torch.empty_like(q).cuda()
    dev = [x.cuda() for x in (q, kc, vc, ks, vs, bt, i32(lens))]
    if decode:
        wllm.paged_attention_decode_block_scaled(out, *dev, hkv, 0.05, BS)
    else:
        wllm.paged_attention_prefill_block_scaled(out, *dev, starts.cuda(), hkv, 0.05, BS)
    got = out.cpu()
    assert torch.equal(got.isnan(), bad)
    zero = torch.zeros((), dtype=dtype)
    K.assert_attention(torch.where(bad, zero, got), ref.masked_fill(bad, 0.0), mag, size, least, dtype, "beside NaN")


def test_prefill_one_short_context():
    check(BF, [50], [20], 4, 2, keys=[(0, 35, 0, 7)], values=[(0, 40, 1, 5)])


@pytest.mark.parametrize("dtype", [BF, F16])
def test_prefill_contexts_that_ctas_share(dtype):
    """Few row blocks behind long contexts: the NaN codes are in some CTAs' parts only."""
    lens, new = [3000, 900, 40], [20, 9, 5]
    check(dtype, lens, new, 4, 2, keys=[(1, 895, 1, 0), (2, 38, 0, 127)],
          values=[(0, 100, 0, 3), (0, 2990, 1, 64), (0, 2999, 0, 127), (1, 500, 0, 65), (2, 0, 1, 0)])


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (7, 1)])
def test_prefill_two_tiles_of_rows(dtype, hq, hkv):
    """Chunks of more than 128 and of more than 256 query rows, where the first rows do not see what the last do."""
    lens, new = [300, 700] + [150] * 160, [60, 200] + [1] * 160  # as many row blocks as SMs: no context is shared
    check(dtype, lens, new, hq, hkv, keys=[(0, 290, 0, 9)], values=[(0, 250, 0, 1), (1, 505, 0, 100), (1, 699, 0, 2), (7, 149, 0, 33)])


@pytest.mark.parametrize("dtype", [BF, F16])
def test_decode_rows_that_ctas_share(dtype):
    check(dtype, [5000, 33, 2000], [1, 1, 1], 8, 2, keys=[(1, 32, 0, 5)],
          values=[(0, 17, 0, 3), (0, 4999, 1, 127), (2, 1000, 0, 64)], decode=True)
