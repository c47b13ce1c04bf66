"""The block-scaled append writes nothing where the packed starts decrease, whatever sequences are valid by themselves."""
import pytest
import torch

import paged_kv_cache_185_gb300 as wllm
from oracle import block_scaled as S
from tests.test_gpu_block_scaled import F16, F32, BF, append_case, i32

pytestmark = pytest.mark.gpu
LENGTHS = 4  # the bit of the error word


def call(case, qsl):
    key, value, ((kc, ks), (vc, vs)), bt, cl, _ = case
    dev = [x.clone().cuda() for x in (kc, vc, ks, vs)]
    wllm.reshape_and_cache_block_scaled(key.cuda(), value.cuda(), *dev, bt.cuda(), cl.cuda(), kc.shape[2], query_start_loc=qsl.cuda())
    return [x.cpu() for x in dev], wllm.device_errors()


def untouched(got, case):
    _, _, ((kc, ks), (vc, vs)), *_ = case
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, (kc, vc, ks, vs)))


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 64), (256, 64)])  # one, two and four warps a block
def test_a_decrease_between_valid_sequences(dtype, d, bs):
    """The span is fine and the first sequence's own start and end are."""
    case = append_case(1, dtype, [20, 33, 16], [4, 0, 12], 2, d, bs)
    assert case[0].shape[0] == 16
    for starts in ([0, 4, 3, 16], [0, 0, -1, 16], [0, 16, 4, 16], [4, 3, 3, 16], [0, 4, 16, 15], [1, 0, 0, 9]):
        got, err = call(case, i32(starts))
        assert err == LENGTHS and untouched(got, case), starts
    got, err = call(case, i32([0, 4, 4, 16]))
    assert err == 0 and not untouched(got, case)


@pytest.mark.parametrize("B", [127, 128, 129, 640, 3000])
def test_wherever_the_decrease_is(B):
    lens, new = [9 + i % 5 for i in range(B)], [1 + i % 3 for i in range(B)]
    case = append_case(B, BF, lens, new, 1, 64, 16)
    good = case[5]
    got, err = call(case, good)
    assert err == 0 and not untouched(got, case)
    for at in (1, 2, B // 2, B - 1):
        starts = good.clone()
        starts[at] = starts[at + 1] + 1
        got, err = call(case, starts)
        assert err == LENGTHS and untouched(got, case), at


def test_a_good_call_behind_a_bad_one():
    case = append_case(5, BF, [20, 33, 16], [4, 17, 16], 2, 128, 16)
    key, value, ((kc, ks), (vc, vs)), bt, cl, qsl = case
    dev = [x.clone().cuda() for x in (kc, vc, ks, vs)]
    rest = [x.cuda() for x in (bt, cl)]
    for starts in (i32([0, 30, 21, 37]), qsl):
        wllm.reshape_and_cache_block_scaled(key.cuda(), value.cuda(), *dev, *rest, 16, query_start_loc=starts.cuda())
    assert wllm.device_errors() == LENGTHS
    ref = [x.clone() for x in (kc, vc, ks, vs)]
    S.append(key, value, *ref, bt, cl, qsl)
    for i, (a, b) in enumerate(zip(dev, ref)):
        a = a.cpu()
        if i < 2:
            same = (a == b) | ((a & 0x7f == 0x7f) & (b & 0x7f == 0x7f))
            assert same.all()
        else:
            assert torch.equal(a.view(torch.int32), b.view(torch.int32))
