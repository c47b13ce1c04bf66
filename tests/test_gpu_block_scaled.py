"""The cache with a scale for each block and head on the GPU: every call against its definition."""
import math
import threading

import pytest
import torch

import oracle
import paged_kv_cache_185_gb300 as wllm
from oracle import block_scaled as S
from tests import block_scaled_helpers as K
from tests import sparse_helpers as H

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
I32, I64 = torch.int32, torch.int64


@pytest.fixture(autouse=True)
def _no_errors():
    wllm.device_errors()
    yield
    assert wllm.device_errors() == 0


def i32(x):
    return torch.tensor(x, dtype=I32)


# ---------------------------------------------------------------- slots
def assign(table, lens, new, stack, count, rows, bs, positions=True, in_place=True):
    """The call on copies on the GPU; (slots, positions, starts, lengths, count, tables, stack) on the host."""
    dev = [x.cuda() for x in (table, lens, new, stack, i32([count]))]
    out = dict(slot_mapping=torch.full((rows,), 77, dtype=I64, device="cuda"), query_start_loc=torch.full((len(lens) + 1,), 77, dtype=I32, device="cuda"))
    pos = torch.full((rows,), 77, dtype=I64, device="cuda") if positions else None
    more = {} if in_place else dict(context_lens_out=torch.full_like(dev[1], 77), num_free_out=torch.full_like(dev[4], 77))
    wllm.assign_slots(out["slot_mapping"], out["query_start_loc"], *dev, bs, positions=pos, **more)
    if not in_place:
        assert torch.equal(dev[1].cpu(), lens) and int(dev[4]) == count
    got = (out["slot_mapping"], pos, out["query_start_loc"], more.get("context_lens_out", dev[1]), more.get("num_free_out", dev[4]), dev[0], dev[3])
    return [None if x is None else x.cpu() for x in got]


def check_assign(table, lens, new, stack, count, rows, bs, **how):
    got = assign(table, lens, new, stack, count, rows, bs, **how)
    ref = S.assign_slots(table, lens, new, stack, count, rows, bs)
    for name, a, b in zip(("slots", "positions", "starts", "lengths", "count", "tables", "stack"), got, ref):
        if a is not None:
            assert torch.equal(a.view(-1), b.view(-1) if torch.is_tensor(b) else i32([b])), name
    return got


def slot_inputs(seed, B, hi, most_new, bs, width=None, ended=0.1, room=60, spare=40):
    g = H.gen(seed)
    lens = torch.randint(0, hi + 1, (B,), generator=g)
    new = torch.randint(0, most_new + 1, (B,), generator=g)
    new[torch.rand(B, generator=g) < ended] = -1
    width = int((hi + most_new) // bs + 1) if width is None else width
    table, pool = H.block_tables(g, lens.tolist(), bs, width=width)
    held = int((-(-lens // bs)).sum())
    stack = torch.full((held + spare + room,), -9, dtype=I32)
    stack[:spare] = 100_000 + torch.randperm(spare, generator=g).to(I32)
    return table, lens.to(I32), new.to(I32), stack, spare


@pytest.mark.parametrize("B,hi,most_new,bs,rows", [
    (1, 0, 1, 16, 1), (1, 40, 1, 16, 4), (3, 20, 5, 8, 40), (32, 300, 1, 16, 32), (33, 64, 20, 32, 700),
    (200, 500, 1, 16, 256), (257, 100, 90, 8, 9000), (1024, 50, 2, 16, 2100), (1025, 50, 2, 16, 2100), (3001, 30, 3, 64, 5000),
    (5, 2000, 2500, 256, 9001), (64, 10, 0, 1, 3), (40, 0, 1500, 32, 40000)])
@pytest.mark.parametrize("in_place", [True, False])
def test_slots(B, hi, most_new, bs, rows, in_place):
    args = slot_inputs(B + hi + bs, B, hi, most_new, bs)
    check_assign(*args, rows, bs, in_place=in_place)
    check_assign(args[0], args[1], args[2].clamp(min=0), *args[3:], rows, bs, in_place=in_place)  # none has ended
    check_assign(args[0], args[1], torch.full_like(args[2], -1), *args[3:], rows, bs, in_place=in_place)  # all have


@pytest.mark.parametrize("spare", [0, 1, 7, 30, 31, 500])
@pytest.mark.parametrize("rows", [0, 1, 60, 400])
def test_slots_run_short(spare, rows):
    args = slot_inputs(5, 50, 60, 12, 8, ended=0.05, spare=spare)
    got = check_assign(*args, rows, 8, positions=False)
    asked = int(args[2].clamp(min=0).sum())
    assert (int(got[2][-1]) < asked) == (rows < asked or spare < 30)


def test_slots_of_no_sequence():
    got = assign(torch.zeros(0, 4, dtype=I32), i32([]), i32([]), i32([5, 6]), 2, 6, 16)
    assert got[0].tolist() == [-1] * 6 and got[2].tolist() == [0] and int(got[4]) == 2


def test_slots_of_the_most_sequences():
    check_assign(*slot_inputs(9, 16384, 9, 1, 16, spare=3000), 16384, 16)


def test_slots_step_after_step():
    """A server's life: sequences begin, grow and end; no block is ever held twice and none is lost."""
    g, bs, B, F = H.gen(3), 4, 12, 60
    table, lens = torch.full((B, 20), -1, dtype=I32), torch.zeros(B, dtype=I32)
    stack, count = torch.randperm(F, generator=g).to(I32), F
    for step in range(25):
        new = torch.randint(0, 9, (B,), generator=g).to(I32)
        new[torch.rand(B, generator=g) < 0.15] = -1
        slots, _, starts, lens, left, table, stack = check_assign(table, lens, new, stack, count, 50, bs)
        count = int(left)
        held = [int(table[b, k]) for b in range(B) for k in range(-(-int(lens[b]) // bs))]
        assert sorted(held + stack[:count].tolist()) == list(range(F)), step


def test_slots_table_rows_with_a_stride():
    table, lens, new, stack, count = slot_inputs(4, 20, 60, 10, 8)
    wide = torch.full((20, 2 * table.shape[1] + 3), -5, dtype=I32).cuda()
    view = wide[:, :table.shape[1]]
    view.copy_(table)
    slots, starts = torch.empty(300, dtype=I64, device="cuda"), torch.empty(21, dtype=I32, device="cuda")
    wllm.assign_slots(slots, starts, view, lens.cuda(), new.cuda(), stack.cuda(), i32([count]).cuda(), 8)
    ref = S.assign_slots(table, lens, new, stack, count, 300, 8)
    assert torch.equal(slots.cpu(), ref[0]) and torch.equal(view.cpu(), ref[5]) and (wide[:, table.shape[1]:] == -5).all()


def test_slots_record_what_is_out_of_range():
    bs = 8
    table, stack = torch.arange(20, dtype=I32).view(4, 5), torch.arange(100, 110, dtype=I32)
    good = [i32([3, 8, 20, 0]), i32([2, 1, 4, 7])]

    def call(lens, new, tab=table, count=10, room=10):
        got = assign(tab, lens, new, stack[:room], count, 40, bs)
        return got, wllm.device_errors()

    assert call(*good)[1] == 0
    for bad in (-1, 41, 2 ** 31 - 1):                      # a length out of range is not served and stays
        lens = good[0].clone()
        lens[1] = bad
        got, err = call(lens, good[1])
        assert err == 4 and int(got[3][1]) == bad and (got[2][1:] - got[2][:-1]).tolist() == [2, 0, 4, 7]
        new = good[1].clone()
        new[1] = -1                                       # nor does it give back anything
        got, err = call(lens, new)
        assert err == 4 and int(got[4]) == 9                # the fourth took one
    new = good[1].clone()
    new[2] = 21                                           # 41 tokens of 40
    got, err = call(good[0], new)
    assert err == 4 and (got[2][1:] - got[2][:-1]).tolist() == [2, 1, 0, 7]
    new[2] = 2 ** 31 - 1
    assert call(good[0], new)[1] == 4
    assert call(*good, count=11)[1] == 4                  # more free blocks than the stack has room for
    got, err = call(*good, count=-3)
    assert err == 4 and int(got[4]) == 0
    got, err = call(good[0], i32([-1, -1, 1, 1]), count=9)  # one place left for two blocks
    assert err == 4
    tab = table.clone()
    tab[0, 0] = -7                                        # the block of tokens 0 .. 7
    got, err = call(*good, tab=tab)
    assert err == 2 and got[0][:2].tolist() == [-1, -1] and (got[0][2:14] >= 0).all()


# ---------------------------------------------------------------- append
def append_case(seed, dtype, lens, new, hkv, d, bs, starts=True, layout="plain", spread=1.0, width=None):
    """Inputs of one append: codes and scales that earlier tokens left, NaN behind them."""
    g = H.gen(seed)
    bt, blocks = H.block_tables(g, lens, bs, width=width)
    before = [n - m for n, m in zip(lens, new)]
    cache = [K.pool(g, blocks, hkv, bs, d, bt, before, spread=1.5) for _ in range(2)]
    rows = len(lens) if not starts else sum(new)
    size = torch.exp2((torch.randn(rows, hkv, 1, generator=g) * spread).round() - 1)
    if layout == "fused":
        both = H.randn(g, rows, 3 * hkv, d) * torch.cat([size] * 3, 1)
        both = both.to(dtype)
        key, value = both[:, hkv:2 * hkv], both[:, 2 * hkv:]
    elif layout == "odd":  # rows that begin at any element
        both = (H.randn(g, rows, hkv, 2 * d + 3) * size).to(dtype)
        key, value = both[:, :, 1:d + 1], both[:, :, d + 2:2 * d + 2]
    else:
        key, value = ((H.randn(g, rows, hkv, d) * size).to(dtype) for _ in range(2))
    qsl = i32([0] + torch.tensor(new).cumsum(0).tolist()) if starts else None
    return key, value, cache, bt, i32(lens), qsl


def on_gpu(x):
    """A copy on the GPU with the same strides."""
    base = torch.empty(x.untyped_storage().size() // x.element_size(), dtype=x.dtype)
    base.set_(x.untyped_storage())
    return base.cuda().as_strided(x.shape, x.stride(), x.storage_offset())


def check_append(key, value, cache, bt, lens, qsl, what=""):
    (kc, ks), (vc, vs) = cache
    dev = [x.clone().cuda() for x in (kc, vc, ks, vs)]
    bs = kc.shape[2]
    wllm.reshape_and_cache_block_scaled(on_gpu(key), on_gpu(value), *dev, bt.cuda(), lens.cuda(), bs,
                                        query_start_loc=None if qsl is None else qsl.cuda())
    ref = [x.clone() for x in (kc, vc, ks, vs)]
    S.append(key, value, ref[0], ref[1], ref[2], ref[3], bt, lens, qsl)
    got = [x.cpu() for x in dev]
    for name, a, b in zip(("k_scales", "v_scales"), got[2:], ref[2:]):
        assert torch.equal(a.view(I32), b.view(I32)), f"{what} {name}"
    for name, a, b in zip(("k_cache", "v_cache"), got[:2], ref[:2]):
        K.same_codes(a, b, f"{what} {name}")
    return got


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("d,bs", [(64, 8), (64, 64), (128, 16), (128, 32), (128, 128), (256, 8), (256, 16), (256, 256)])
def test_append_chunks(dtype, d, bs):
    lens = [1, bs - 1, bs, bs + 1, 2 * bs + 3, 5 * bs, 3 * bs + 2, 40, 0, 4 * bs + 5]
    new = [1, bs - 1, bs, 1, bs + 2, 3 * bs, 3 * bs + 2, 0, 0, 2 * bs]
    check_append(*append_case(d + bs, dtype, lens, new, 2, d, bs))


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("d,bs,hkv", [(64, 16, 3), (128, 16, 8), (128, 8, 1), (256, 64, 2)])
def test_append_one_token(dtype, d, bs, hkv):
    lens = [1, 2, bs, bs + 1, 0, 3 * bs, 3 * bs + 1, 7, 0] + list(range(bs, 2 * bs + 1, 3))
    got = check_append(*append_case(d, dtype, lens, [min(n, 1) for n in lens], hkv, d, bs, starts=False))
    assert len(got) == 4


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("layout", ["fused", "odd"])
@pytest.mark.parametrize("starts", [True, False])
def test_append_strided_rows(dtype, layout, starts):
    lens = [30, 17, 1, 64]
    check_append(*append_case(3, dtype, lens, [13, 1, 1, 50] if starts else [1] * 4, 2, 128, 16, starts=starts, layout=layout))


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("starts", [True, False])
@pytest.mark.parametrize("bs", [8, 16, 64])
def test_append_odd_values(dtype, starts, bs):
    """Zeros, infinities, NaN, the type's largest and least values; scales that do not rise, rise a little, and far."""
    lens, new = [bs + 5] * 9, ([3] * 9 if starts else [1] * 9)
    key, value, cache, bt, cl, qsl = append_case(7, dtype, lens, new, 2, 128, bs, starts=starts)
    step = new[0]
    big, small = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    for i, x in enumerate((0.0, math.inf, math.nan, big, small, 448 * 2.0 ** -6, 448 * 2.0 ** -6 * (1 + 2.0 ** -7), -math.inf)):
        key[i * step:(i + 1) * step] = 0.0
        key[i * step, :, 5] = x
        key[i * step, :, 6] = -1.5 if i != 4 else 0.0
        value[i * step] = x
    check_append(key, value, cache, bt, cl, qsl)


def test_append_scales_that_are_no_powers_of_two():
    key, value, cache, bt, cl, qsl = append_case(11, BF, [20, 27, 30, 18, 19, 25], [3] * 6, 2, 128, 16)
    for _, s in cache:
        s.copy_(torch.where(s.isnan(), s, s * 0.7))
        s[bt[3, 1]] = 0.0        # what no append writes counts as the nearer end of the range
        s[bt[4, 1]] = math.nan
        s[bt[5, 1]] = 2.0 ** 60
    check_append(key, value, cache, bt, cl, qsl)


def test_append_twice_is_once():
    key, value, cache, bt, cl, qsl = append_case(12, BF, [20, 50, 16], [3, 40, 16], 4, 128, 16)
    once = check_append(key, value, cache, bt, cl, qsl)
    twice = check_append(key, value, [(once[0], once[2]), (once[1], once[3])], bt, cl, qsl)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(once, twice))


def test_append_in_pieces_holds_the_values():
    """Token by token the codes are those of one append, but for values that a rise brought below the normal codes."""
    g, n, hkv, d, bs = H.gen(13), 48, 2, 128, 16
    key = (H.randn(g, n, hkv, d) * torch.exp2(torch.arange(n) / 4.0)[:, None, None]).to(BF)
    bt = i32([[2, 0, 1]])
    caches = [torch.zeros(3, hkv, bs, d, dtype=torch.uint8, device="cuda") for _ in range(4)]
    scales = [torch.full((3, hkv), math.nan, device="cuda") for _ in range(4)]
    wllm.reshape_and_cache_block_scaled(key.cuda(), key.cuda(), caches[0], caches[1], scales[0], scales[1], bt.cuda(), i32([n]).cuda(),
                                        bs, query_start_loc=i32([0, n]).cuda())
    for t in range(n):
        wllm.reshape_and_cache_block_scaled(key[t:t + 1].cuda(), key[t:t + 1].cuda(), caches[2], caches[3], scales[2], scales[3],
                                            bt.cuda(), i32([t + 1]).cuda(), bs)
    assert torch.equal(scales[0], scales[2]) and torch.equal(scales[1], scales[3]) and torch.equal(scales[0], scales[1])
    a, b = (oracle.widen_e4m3(c.cpu()) for c in (caches[0], caches[2]))
    # each rise rounds to a multiple of 2^-9 of the new scale: off by 2^-10, halved by every rise after it
    assert ((a - b).abs() <= torch.where(a.abs() >= 2.0 ** -6, 0.0, 2 * 2.0 ** -10)).all()
    assert (a != b).any()


def test_append_records_what_is_out_of_range():
    key, value, cache, bt, cl, qsl = append_case(14, BF, [20, 33, 16], [4, 17, 16], 2, 64, 16)
    (kc, ks), (vc, vs) = cache

    def call(cl=cl, qsl=qsl, bt=bt):
        dev = [x.clone().cuda() for x in (kc, vc, ks, vs)]
        wllm.reshape_and_cache_block_scaled(key.cuda(), value.cuda(), *dev, bt.cuda(), cl.cuda(), 16, query_start_loc=qsl.cuda())
        return [x.cpu() for x in dev], wllm.device_errors()

    def untouched(got):
        return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, (kc, vc, ks, vs)))

    assert call()[1] == 0
    assert call(cl=i32([20, 16, 16]))[1] == 4             # 17 new tokens of 16
    assert call(cl=i32([20, 33, 49]))[1] == 4             # more than the table's row has
    assert call(cl=i32([20, -1, 16]))[1] == 4
    for bad in ([0, 4, 21, 38], [0, 4, 21, 3 * 48 + 1], [30, 4, 21, 4], [0, 4, 21, -5]):
        got, err = call(qsl=i32(bad))
        assert err == 4 and untouched(got), bad
    assert call(qsl=i32([0, 21, 4, 37]))[1] & 4           # decreasing
    for bad in (-1, kc.shape[0], 2 ** 31 - 1):
        b2 = bt.clone()
        b2[1, 1] = bad
        got, err = call(bt=b2)
        ref = [x.clone() for x in (kc, vc, ks, vs)]
        S.append(key[:4], value[:4], *ref, bt[:1], cl[:1], i32([0, 4]))
        i = bt[0, 1]
        assert err == 2 and torch.equal(got[0][i], ref[0][i])


# ---------------------------------------------------------------- decode
def attention_case(seed, dtype, lens, hq, hkv, d, bs, rows=None, spread=0.5, width=None, q_scale=1.0):
    g = H.gen(seed)
    bt, blocks = H.block_tables(g, lens, bs, width=width)
    kc, ks = K.pool(g, blocks, hkv, bs, d, bt, lens, spread)
    vc, vs = K.pool(g, blocks, hkv, bs, d, bt, lens, spread)
    q = H.randn(g, len(lens) if rows is None else rows, hq, d, dtype=dtype, scale=q_scale)
    return q, kc, vc, ks, vs, bt, i32(lens)


def check_decode(q, kc, vc, ks, vs, bt, cl, scale, what="", layout="plain", workspace=None):
    bs, hkv = kc.shape[2], kc.shape[1]
    if layout == "odd":
        qd = torch.zeros(q.shape[0], q.shape[1], q.shape[2] + 3, dtype=q.dtype, device="cuda")[:, :, 1:q.shape[2] + 1]
        qd.copy_(q)
        out = torch.zeros(q.shape[0], q.shape[1] + 1, q.shape[2] + 5, dtype=q.dtype, device="cuda")[:, 1:, 3:q.shape[2] + 3]
    else:
        qd, out = q.cuda(), torch.full_like(q, 9.0).cuda()
    wllm.paged_attention_decode_block_scaled(out, qd, *(x.cuda() for x in (kc, vc, ks, vs, bt, cl)), hkv, scale, bs, workspace=workspace)
    ref, mag, size, least = S.attention(q, kc, vc, ks, vs, bt, cl, scale)
    K.assert_attention(out.cpu(), ref, mag, size, least, q.dtype, what)
    return out


SHAPES = [(4, 4, 64, 16), (8, 2, 64, 32), (7, 1, 128, 16), (8, 1, 128, 8), (14, 2, 128, 64), (16, 1, 128, 16), (20, 1, 64, 16),
          (33, 1, 128, 16), (3, 3, 256, 16), (12, 1, 256, 8), (8, 8, 128, 256)]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
def test_decode(dtype, hq, hkv, d, bs):
    lens = [1, 0, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 0, 300, 2]
    case = attention_case(hq + d + bs, dtype, lens, hq, hkv, d, bs)
    out = check_decode(*case, 1.0 / math.sqrt(d))
    assert not out[1].any() and not out[15].any()


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("lens", [[5000], [4000, 1, 0, 3000], [257] * 40])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (8, 2, 128), (16, 1, 128), (2, 2, 256)])
def test_decode_rows_that_ctas_share(dtype, lens, hq, hkv, d):
    check_decode(*attention_case(len(lens) + d, dtype, lens, hq, hkv, d, 16), 1.0 / math.sqrt(d))


@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-6])
def test_decode_scales_of_the_score(scale):
    check_decode(*attention_case(2, BF, [40, 1, 1000], 4, 2, 128, 16), scale)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("spread", [3.0, 12.0])
def test_decode_blocks_of_very_unequal_scales(dtype, spread):
    """Scales as far apart as the range allows; the scores stay moderate."""
    q, kc, vc, ks, vs, bt, cl = attention_case(8, dtype, [200, 33, 700], 8, 2, 128, 16, spread=spread)
    ks = torch.where(ks.isnan(), ks, ks.clamp(max=2.0 ** -5))
    check_decode(q, kc, vc, ks, vs if dtype == BF else vs.clamp(max=2.0 ** 4), bt, cl, 0.05)


def test_decode_scales_out_of_range_count_as_its_ends():
    q, kc, vc, ks, vs, bt, cl = attention_case(9, BF, [50, 40], 4, 2, 128, 16)
    ks[bt[0, 0]] = 0.0
    ks[bt[0, 1]] = 2.0 ** -60
    vs[bt[0, 2]] = -1.0
    vs[bt[1, 0]] = 2.0 ** 70
    check_decode(q, kc, vc, ks, vs, bt, cl, 0.05)
    ks[bt[0, 0]] = math.nan
    out = check_decode(q, kc, vc, ks.nan_to_num(nan=0.0), vs.nan_to_num(nan=0.0), bt, cl, 0.05)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("q_scale", [1e-30, 1e-4, 1e4, 1e30])
def test_decode_queries_of_any_size(q_scale):
    """bf16 queries far outside f16's range; the scale brings the scores back."""
    check_decode(*attention_case(10, BF, [50, 40, 333], 4, 2, 128, 16, q_scale=q_scale), 0.05 / q_scale)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_rows_of_any_alignment(dtype, d):
    check_decode(*attention_case(11, dtype, [50, 0, 333], 6, 2, d, 16), 0.05, layout="odd")


def test_decode_not_a_number_where_it_belongs():
    q, kc, vc, ks, vs, bt, cl = attention_case(12, BF, [50, 40], 4, 2, 128, 16)
    kc[bt[0, 1], 0, 3, 7] = K.NAN_CODE   # a key of sequence 0, kv head 0
    vc[bt[1, 0], 1, 2, 5] = K.NAN_CODE   # a value element of sequence 1, kv head 1
    out = torch.empty_like(q).cuda()
    wllm.paged_attention_decode_block_scaled(out, q.cuda(), *(x.cuda() for x in (kc, vc, ks, vs, bt, cl)), 2, 0.05, 16)
    nan = out.isnan().cpu()
    assert nan[0, :2].all() and not nan[0, 2:].any() and nan[1, 2:, 5].all() and int(nan[1].sum()) == 2


@pytest.mark.parametrize("B", [129, 1000, 2500])
def test_decode_many_sequences(B):
    g = H.gen(B)
    lens = torch.randint(0, 40, (B,), generator=g).tolist()
    check_decode(*attention_case(B, BF, lens, 4, 2, 64, 16), 0.1)


def test_decode_is_the_same_every_time():
    case = attention_case(14, BF, [3000, 70, 2000, 0, 900], 8, 2, 128, 16)
    a = check_decode(*case, 0.08)
    for _ in range(5):
        assert torch.equal(a, check_decode(*case, 0.08))


def test_decode_wide_tables_and_entries_behind_the_end():
    q, kc, vc, ks, vs, bt, cl = attention_case(15, BF, [50, 40], 4, 2, 128, 16, width=3000)
    bt[:, 5:] = 2 ** 31 - 1
    check_decode(q, kc, vc, ks, vs, bt, cl, 0.05)


def test_decode_records_what_is_out_of_range():
    q, kc, vc, ks, vs, bt, cl = (x.cuda() for x in attention_case(16, BF, [50, 40, 30], 4, 2, 128, 16))
    out = torch.empty_like(q)
    good = wllm.paged_attention_decode_block_scaled(out, q, kc, vc, ks, vs, bt, cl, 2, 0.05, 16).clone()
    assert wllm.device_errors() == 0
    for bad in (-1, kc.shape[0], 2 ** 31 - 1):
        b2 = bt.clone()
        b2[1, 1] = bad
        wllm.paged_attention_decode_block_scaled(out, q, kc, vc, ks, vs, b2, cl, 2, 0.05, 16)
        assert wllm.device_errors() == 2 and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    for bad in (-1, 65, 2 ** 31 - 1):
        c2 = cl.clone()
        c2[1] = bad
        b2 = bt.clamp(min=0)
        wllm.paged_attention_decode_block_scaled(out, q, kc, vc, ks, vs, b2, c2, 2, 0.05, 16)
        assert wllm.device_errors() == 4 and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


def test_decode_beyond_32_bits():
    """Blocks whose codes lie more than 2^32 bytes into the pool."""
    blocks, hkv, bs, d = 150_000, 2, 128, 128  # 4.9 GB
    g = H.gen(17)
    small = attention_case(17, BF, [300, 500], 4, hkv, d, bs)
    q, kc, vc, ks, vs, bt, cl = small
    far = blocks - kc.shape[0]
    assert far * hkv * bs * d > 2 ** 32
    big = [torch.zeros(blocks, hkv, bs, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(blocks, hkv, device="cuda") for _ in range(2)]
    for x, y in zip(big + scales, (kc, vc, ks, vs)):
        x[far:] = y.cuda()
    out = torch.empty_like(q).cuda()
    moved = torch.where(bt >= 0, bt + far, bt).cuda()
    wllm.paged_attention_decode_block_scaled(out, q.cuda(), *big, *scales, moved, cl.cuda(), hkv, 0.05, bs)
    K.assert_attention(out.cpu(), *S.attention(q, kc, vc, ks, vs, bt, cl, 0.05), BF, "far blocks")
    qp = H.randn(g, 40, 4, d, dtype=BF)
    starts = i32([0, 25, 40])
    outp = torch.empty_like(qp).cuda()
    wllm.paged_attention_prefill_block_scaled(outp, qp.cuda(), *big, *scales, moved, cl.cuda(), starts.cuda(), hkv, 0.05, bs)
    K.assert_attention(outp.cpu(), *S.attention(qp, kc, vc, ks, vs, bt, cl, 0.05, starts), BF, "far blocks, chunks")
    key = H.randn(g, 2, hkv, d, dtype=BF)
    wllm.reshape_and_cache_block_scaled(key.cuda(), key.cuda(), *big, *scales, moved, cl.cuda(), bs)
    ref = [x.clone() for x in (kc, vc, ks, vs)]
    S.append(key, key, *ref, bt, cl)
    K.same_codes(big[0][far:].cpu(), ref[0], "far blocks, append")
    assert torch.equal(scales[1][far:].cpu().view(I32), ref[3].view(I32))


# ---------------------------------------------------------------- prefill
def check_prefill(q, kc, vc, ks, vs, bt, cl, starts, scale, layout="plain", what=""):
    bs, hkv = kc.shape[2], kc.shape[1]
    if layout == "odd":
        qd = torch.zeros(q.shape[0], q.shape[1], q.shape[2] + 3, dtype=q.dtype, device="cuda")[:, :, 1:q.shape[2] + 1]
        qd.copy_(q)
        out = torch.zeros(q.shape[0], q.shape[1] + 1, q.shape[2] + 5, dtype=q.dtype, device="cuda")[:, 1:, 3:q.shape[2] + 3]
    else:
        qd, out = q.cuda(), torch.full_like(q, 9.0).cuda()
    wllm.paged_attention_prefill_block_scaled(out, qd, *(x.cuda() for x in (kc, vc, ks, vs, bt, cl, starts)), hkv, scale, bs)
    ref, mag, size, least = S.attention(q, kc, vc, ks, vs, bt, cl, scale, starts)
    rows = int(starts[-1])
    K.assert_attention(out[:rows].cpu(), ref[:rows], mag[:rows], size[:rows], least[:rows], q.dtype, what)
    assert layout == "odd" or (out[rows:] == 9.0).all()
    return out


def chunks(lens, new, pad=0):
    starts = i32([0] + torch.tensor(new).cumsum(0).tolist())
    return starts, int(starts[-1]) + pad


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("hq,hkv,d,bs", [s for s in SHAPES if s[2] < 256])
def test_prefill(dtype, hq, hkv, d, bs):
    lens = [1, 0, 5, 127, 128, 129, 40, 300, 64, 200]
    new = [1, 0, 5, 127, 3, 129, 0, 1, 40, 150]
    starts, rows = chunks(lens, new, pad=2)
    check_prefill(*attention_case(hq + d + bs, dtype, lens, hq, hkv, d, bs, rows=rows), starts, 1.0 / math.sqrt(d))


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 16), (128, 8)])
def test_prefill_long(dtype, d, bs):
    lens, new = [1500, 900], [700, 257]
    starts, rows = chunks(lens, new)
    check_prefill(*attention_case(d, dtype, lens, 6, 2, d, bs, rows=rows), starts, 1.0 / math.sqrt(d))


@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-6])
def test_prefill_scales_of_the_score(scale):
    starts, rows = chunks([40, 1, 400], [40, 1, 30])
    check_prefill(*attention_case(2, BF, [40, 1, 400], 4, 2, 128, 16, rows=rows), starts, scale)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("spread", [3.0, 12.0])
@pytest.mark.parametrize("bs", [8, 16])
def test_prefill_blocks_of_very_unequal_scales(dtype, spread, bs):
    starts, rows = chunks([200, 33, 700], [100, 33, 50])
    q, kc, vc, ks, vs, bt, cl = attention_case(8, dtype, [200, 33, 700], 8, 2, 128, bs, rows=rows, spread=spread)
    ks = torch.where(ks.isnan(), ks, ks.clamp(max=2.0 ** -5))
    check_prefill(q, kc, vc, ks, vs if dtype == BF else vs.clamp(max=2.0 ** 4), bt, cl, starts, 0.05)


@pytest.mark.parametrize("q_scale", [1e-30, 1e-4, 1e4, 1e30])
def test_prefill_queries_of_any_size(q_scale):
    starts, rows = chunks([50, 300], [20, 5])
    check_prefill(*attention_case(10, BF, [50, 300], 4, 2, 128, 16, rows=rows, q_scale=q_scale), starts, 0.05 / q_scale)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_rows_of_any_alignment(dtype, d):
    starts, rows = chunks([50, 0, 333], [20, 0, 100])
    check_prefill(*attention_case(11, dtype, [50, 0, 333], 6, 2, d, 16, rows=rows), starts, 0.05, layout="odd")


@pytest.mark.parametrize("lens,new", [([300], [60]), ([64], [64]), ([65], [1]), ([129], [100]), ([1000, 70, 0, 1], [40, 70, 0, 1])])
@pytest.mark.parametrize("width", [None, 130, 1500])
def test_prefill_contexts_shorter_than_the_tables(lens, new, width):
    """Few row blocks, whose contexts are shared by as many CTAs as they are long, not as the tables are wide."""
    starts, rows = chunks(lens, new)
    check_prefill(*attention_case(70, F16, lens, 4, 1, 128, 16, rows=rows, width=width), starts, 0.08)


def test_prefill_many_sequences():
    g = H.gen(5)
    lens = torch.randint(1, 60, (150,), generator=g).tolist()
    new = [max(0, min(n, n - 20 + i % 25)) for i, n in enumerate(lens)]
    starts, rows = chunks(lens, new)
    check_prefill(*attention_case(6, BF, lens, 4, 2, 64, 16, rows=rows), starts, 0.1)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (7, 1), (35, 5)])  # with one kv head contexts are split between CTAs
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_row_counts_beside_those_of_warps_and_tiles(hq, hkv, d):
    new = [1, 31, 32, 33, 64, 97, 128, 129, 160, 161, 255, 256, 257] if hq == hkv else [5, 4, 18, 19, 36, 37, 55, 10]
    lens = [n + (0, 40, 150, 513)[i % 4] for i, n in enumerate(new)]
    starts, rows = chunks(lens, new, pad=1)
    check_prefill(*attention_case(50 + hq, BF, lens, hq, hkv, d, 16, rows=rows), starts, 1.0 / math.sqrt(d))


@pytest.mark.parametrize("hq,hkv", [(4, 1), (32, 8)])
def test_prefill_is_the_same_every_time(hq, hkv):
    """Alone, beside itself on other streams, and replayed from graphs on two streams at once."""
    lens, new = [900, 40, 2000, 333, 1200], [100, 40, 9, 300, 257]
    starts, rows = chunks(lens, new)
    case = [x.cuda() for x in attention_case(60, BF, lens, hq, hkv, 128, 16, rows=rows)] + [starts.cuda()]

    def run(out):
        return wllm.paged_attention_prefill_block_scaled(out, *case, hkv, 0.08, 16)

    alone = run(torch.empty_like(case[0]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 3]):
            outs.append(run(torch.empty_like(case[0])))
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph, out = torch.cuda.CUDAGraph(), torch.empty_like(case[0])
        with torch.cuda.graph(graph):
            run(out)
            run(out)
        graphs.append(graph), outs.append(out)
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, alone) for o in outs)


def test_prefill_of_one_token_is_the_decode():
    lens = [50, 1, 700, 16]
    q, kc, vc, ks, vs, bt, cl = attention_case(7, BF, lens, 8, 2, 128, 16)
    a = check_decode(q, kc, vc, ks, vs, bt, cl, 0.08).float()
    b = check_prefill(q, kc, vc, ks, vs, bt, cl, i32([0, 1, 2, 3, 4]), 0.08).float()
    assert (a - b).norm() <= 2.0 ** -7 * a.norm()


def test_prefill_not_a_number_where_it_belongs():
    q, kc, vc, ks, vs, bt, cl = attention_case(12, BF, [50], 4, 2, 128, 16, rows=20)
    kc[bt[0, 2], 0, 3, 7] = K.NAN_CODE   # the key of token 35: rows of positions 35 on
    vc[bt[0, 2], 1, 8, 5] = K.NAN_CODE   # a value element of token 40
    out = torch.empty_like(q).cuda()
    wllm.paged_attention_prefill_block_scaled(out, q.cuda(), *(x.cuda() for x in (kc, vc, ks, vs, bt, cl, i32([0, 20]))), 2, 0.05, 16)
    nan = out.isnan().cpu()
    assert nan[5:, :2].all() and not nan[:5].any()
    assert nan[10:, 2:, 5].all() and int(nan[:, 2:].sum()) >= 20 and not nan[:10, 2:].any()


def test_prefill_records_what_is_out_of_range():
    lens, new = [50, 40, 30], [10, 5, 30]
    starts, rows = chunks(lens, new)
    q, kc, vc, ks, vs, bt, cl = (x.cuda() for x in attention_case(16, BF, lens, 4, 2, 128, 16, rows=rows))
    out = torch.zeros_like(q)
    good = wllm.paged_attention_prefill_block_scaled(out, q, kc, vc, ks, vs, bt, cl, starts.cuda(), 2, 0.05, 16).clone()
    assert wllm.device_errors() == 0
    for bad in (-1, kc.shape[0], 2 ** 31 - 1):
        b2 = bt.clone()
        b2[1, 1] = bad
        wllm.paged_attention_prefill_block_scaled(out, q, kc, vc, ks, vs, b2, cl, starts.cuda(), 2, 0.05, 16)
        assert wllm.device_errors() == 2 and torch.equal(out[:10], good[:10]) and torch.equal(out[15:], good[15:])
    for bad in (-1, 4, 65, 2 ** 31 - 1):
        c2 = cl.clone()
        c2[1] = bad
        wllm.paged_attention_prefill_block_scaled(out, q, kc, vc, ks, vs, bt.clamp(min=0), c2, starts.cuda(), 2, 0.05, 16)
        assert wllm.device_errors() == 4 and torch.equal(out[:10], good[:10]) and torch.equal(out[15:], good[15:])
    for bad in ([0, 10, 15, 46], [-1, 10, 15, 45], [0, 16, 15, 45]):
        wllm.paged_attention_prefill_block_scaled(out, q, kc, vc, ks, vs, bt, cl, i32(bad).cuda(), 2, 0.05, 16)
        assert wllm.device_errors() == 4


# ---------------------------------------------------------------- together
class Server:
    """Two layers' caches, tables and free blocks on the GPU, and what was ever appended, on the host."""

    def __init__(self, B, blocks, hkv, d, bs, width, dtype=BF, layers=2):
        self.B, self.hkv, self.d, self.bs, self.dtype = B, hkv, d, bs, dtype
        new = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
        self.caches = [[new(blocks, hkv, bs, d, dtype=torch.uint8) for _ in range(2)] + [new(blocks, hkv) for _ in range(2)] for _ in range(layers)]
        self.table, self.lens = torch.full((B, width), -1, dtype=I32, device="cuda"), new(B, dtype=I32)
        self.free, self.count = torch.arange(blocks, dtype=I32, device="cuda"), torch.full((1,), blocks, dtype=I32, device="cuda")

    def buffers(self, rows, hq):
        x = dict(new=torch.zeros(self.B, dtype=I32), slots=torch.zeros(rows, dtype=I64), positions=torch.zeros(rows, dtype=I64),
                 starts=torch.zeros(self.B + 1, dtype=I32), q=torch.zeros(rows, hq, self.d, dtype=self.dtype),
                 key=torch.zeros(rows, self.hkv, self.d, dtype=self.dtype), out=torch.zeros(rows, hq, self.d, dtype=self.dtype))
        return {k: v.cuda() for k, v in x.items()}

    def step(self, x, scale, decode):
        """One step of every layer, as a model would make it: layer l's query is the one before's output plus its own."""
        wllm.assign_slots(x["slots"], x["starts"], self.table, self.lens, x["new"], self.free, self.count, self.bs, positions=x["positions"])
        for c in self.caches:
            wllm.reshape_and_cache_block_scaled(x["key"], x["key"], *c, self.table, self.lens, self.bs,
                                                query_start_loc=None if decode else x["starts"])
            if decode:
                wllm.paged_attention_decode_block_scaled(x["out"], x["q"], *c, self.table, self.lens, self.hkv, scale, self.bs)
            else:
                wllm.paged_attention_prefill_block_scaled(x["out"], x["q"], *c, self.table, self.lens, x["starts"], self.hkv, scale, self.bs)


def test_a_server_from_prompts_to_the_end():
    """Prompts in chunks, decode steps, ends and new prompts; every output against attention over what was appended."""
    g, B, hq, hkv, d, bs = H.gen(21), 6, 8, 2, 128, 16
    s = Server(B, 60, hkv, d, bs, 20)
    said = [[] for _ in range(B)]  # the keys of each sequence, as appended
    scale = 0.06

    def check(x, news):
        at = 0
        for b, n in enumerate(news):
            if n < 0:
                said[b] = []
                continue
            rows = x["key"][at:at + n].cpu()
            said[b] += list(rows)
            kv = torch.stack(said[b]).double() if said[b] else torch.zeros(0, hkv, d)
            for i in range(n):
                L = len(said[b]) - n + i + 1
                for h in range(hq):
                    k = kv[:L, h // (hq // hkv)]
                    ref = torch.softmax(k @ x["q"][at + i, h].cpu().double() * scale, 0) @ k
                    got = x["out"][at + i, h].cpu().double()
                    # E4M3: half a step 2^-4 of each value, in keys and values alike
                    assert (got - ref).norm() <= 0.09 * k.norm(dim=1).max(), (b, i, h)
            at += n
        assert torch.equal(s.lens.cpu(), i32([len(t) for t in said]))

    for news in ([20, 0, 7, 33, 0, 1], [16, 40, 1, 1, 5, 1], [1] * 6, [-1, 1, 1, -1, 1, 1], [30, 1, 1, 17, 1, 1]):
        x = s.buffers(sum(max(n, 0) for n in news), hq)
        x["new"].copy_(i32(news))
        x["q"].copy_(H.randn(g, *x["q"].shape, dtype=BF))
        x["key"].copy_(H.randn(g, *x["key"].shape, dtype=BF))
        s.step(x, scale, decode=all(n == 1 for n in news))
        check(x, news)


def test_captured_steps():
    """Whole decode steps captured and replayed follow the eager ones bit for bit; two graphs on two streams at once."""
    g, B, hq, hkv, d, bs = H.gen(22), 9, 8, 2, 128, 16

    def fresh():
        s = Server(B, 3000, hkv, d, bs, 320)
        x = s.buffers(4000, hq)
        h = H.gen(5)
        x["new"].copy_(i32([1500, 3, 40, 900, 16, 15, 1, 200, 1100]))
        x["key"].copy_(H.randn(h, *x["key"].shape, dtype=BF))
        x["q"].copy_(H.randn(h, *x["q"].shape, dtype=BF))
        s.step(x, 0.06, decode=False)
        y = s.buffers(B, hq)
        y["new"].fill_(1)
        return s, y

    inputs = [(H.randn(g, B, hq, d, dtype=BF).cuda(), H.randn(g, B, hkv, d, dtype=BF).cuda()) for _ in range(6)]
    s, x = fresh()
    ref = []
    for q, key in inputs:
        x["q"].copy_(q), x["key"].copy_(key)
        s.step(x, 0.06, decode=True)
        ref.append(x["out"].clone())
    graphs = []
    for _ in range(2):
        s, x = fresh()
        x["q"].copy_(inputs[0][0]), x["key"].copy_(inputs[0][1])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step(x, 0.06, decode=True)
        graphs.append((graph, s, x, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i, (q, key) in enumerate(inputs):
        for graph, s, x, stream in graphs:
            with torch.cuda.stream(stream):
                x["q"].copy_(q), x["key"].copy_(key)
                graph.replay()
        torch.cuda.synchronize()
        for graph, s, x, stream in graphs:
            assert torch.equal(x["out"], ref[i]), i


def test_streams_and_threads_at_once():
    """Decodes of long rows on several streams, from several threads, share nothing."""
    cases = [attention_case(30 + i, BF, [3000 + 500 * i, 40, 2000], 8, 2, 128, 16) for i in range(4)]
    dev = [[x.cuda() for x in c] for c in cases]
    alone = [wllm.paged_attention_decode_block_scaled(torch.empty_like(c[0]), *c, 2, 0.08, 16) for c in dev]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(c[0]) for _ in range(20)] for c in dev]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for out in outs[i]:
                wllm.paged_attention_decode_block_scaled(out, *dev[i], 2, 0.08, 16)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads], [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in range(4):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


def test_a_workspace_of_the_callers():
    ws = wllm.block_scaled_workspace()
    case = attention_case(40, BF, [3000, 40], 8, 2, 128, 16)
    for fill in (0, 255, 1):  # what is in it does not matter
        check_decode(*case, 0.08, workspace=ws.fill_(fill))
    for bad in (ws[:-1], ws[1:], ws[::2]):
        with pytest.raises(wllm.WllmError):
            check_decode(*case, 0.08, workspace=bad)


def test_slots_of_more_rows_than_a_round_takes():
    """Rows and table entries beyond what every thread of the call has one of."""
    table, lens, new, stack, count = slot_inputs(70, 300, 900, 700, 8, room=130000, spare=40000)
    check_assign(table, lens, new, stack, count, 90000, 8)


def test_check_mode(monkeypatch):
    monkeypatch.setenv("WLLM_CHECK", "1")
    q, kc, vc, ks, vs, bt, cl = attention_case(16, BF, [50, 40], 4, 2, 128, 16)
    check_decode(q, kc, vc, ks, vs, bt, cl, 0.05)
    bt[0, 0] = -1
    with pytest.raises(wllm.WllmError) as e:
        check_decode(q, kc, vc, ks, vs, bt, cl, 0.05)
    assert e.value.status == 3
    with pytest.raises(wllm.WllmError):
        assign(torch.zeros(1, 2, dtype=I32), i32([99]), i32([1]), i32([1, 2]), 2, 4, 16)
