"""Attention over a block-scaled cache where query rows, scales and the score's scale are as large as they may be."""
import pytest
import torch

import paged_kv_cache_185_gb300 as wllm
from oracle import block_scaled as S
from tests import block_scaled_helpers as K
from tests import sparse_helpers as H

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("q_size,scale", [(3e38, 0.05), (3e38, -3e38), (1.0, 3e38), (1e-38, 1.0)])
def test_keys_of_zero_weigh_the_same(form, q_size, scale):
    """Scores of zero are zero whatever they are multiplied with: the output is the mean of the values."""
    g, lens, bs, hkv, d = H.gen(1), [40, 5, 300], 16, 2, 128
    bt, blocks = H.block_tables(g, lens, bs)
    kc, ks = K.pool(g, blocks, hkv, bs, d, bt, lens)
    vc, vs = K.pool(g, blocks, hkv, bs, d, bt, lens)
    kc = torch.where(kc == K.NAN_CODE, kc, torch.zeros_like(kc))
    ks = torch.where(ks.isnan(), ks, torch.full_like(ks, 2.0 ** 40))
    q = (H.randn(g, 3, 4, d).sign() * q_size).to(BF)
    starts = (i32([0, 1, 2, 3]),) if form == "prefill" else ()
    out = torch.empty_like(q).cuda()
    dev = [x.cuda() for x in (q, kc, vc, ks, vs, bt, i32(lens), *starts)]
    call = wllm.paged_attention_prefill_block_scaled if form == "prefill" else wllm.paged_attention_decode_block_scaled
    call(out, *dev, hkv, scale, bs)
    ref, mag, size, least = S.attention(q, kc, vc, ks, vs, bt, i32(lens), scale, *starts)
    assert not size.any()
    K.assert_attention(out.cpu(), ref, mag, size, least, BF, form)
    assert wllm.device_errors() == 0
