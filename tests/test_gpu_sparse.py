"""Key bounds, block selection and block-sparse decode on the GPU against their binary64 definitions, alone and as the
steps of a decode over a growing cache, captured, on two streams and in threads."""
import math
import threading

import pytest
import torch

import oracle
import paged_kv_cache_185_gb300 as wllm
from oracle import sparse as S
from tests import sparse_helpers as H

pytestmark = pytest.mark.gpu
BF, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def cuda(*xs):
    return [None if x is None else x.cuda() for x in xs]


# ---------------------------------------------------------------- bounds
def run_bounds(kb, kc, bt, cl, qsl=None):
    kbd, kcd, btd, cld, qd = cuda(kb, kc, bt, cl, qsl)
    assert wllm.update_key_bounds(kbd, kcd, btd, cld, kc.shape[2], query_start_loc=qd) is kbd
    torch.cuda.synchronize()
    return kbd.cpu()


def assert_bounds(got, kb, kc, bt, cl, new):
    ref = S.key_bounds(kc, bt, cl, new, S.values(kb))
    assert torch.equal(S.values(got).nan_to_num(1e30), ref.nan_to_num(1e30))


@pytest.mark.parametrize("dtype", [F32, F16, BF, U8])
@pytest.mark.parametrize("D,bs,Hkv", [(64, 8, 3), (64, 16, 1), (128, 16, 4), (128, 64, 2), (256, 32, 1), (256, 8, 2), (128, 256, 1)])
def test_bounds_of_chunks_and_steps(dtype, D, bs, Hkv):
    g = H.gen(D + bs)
    lens = [1, bs - 1, bs, bs + 1, 5 * bs, 3 * bs + 2, 0, 9 * bs, 2 * bs]
    new = [1, bs - 1, 1, 2, 5 * bs, bs + 3, 0, 4 * bs + 1, 0]
    bt, pool = H.block_tables(g, lens, bs)
    kc = H.cache(g, pool, Hkv, bs, D, dtype, bt, lens)
    kb = H.cache(g, pool, Hkv, 2, D, dtype)
    qsl = i32([0] + new).cumsum(0).to(torch.int32)
    assert_bounds(run_bounds(kb, kc, bt, i32(lens), qsl), kb, kc, bt, i32(lens), new)
    step = [1 if n else 0 for n in lens]
    assert_bounds(run_bounds(kb, kc, bt, i32(lens)), kb, kc, bt, i32(lens), step)
    assert wllm.device_errors() == 0


def test_bounds_of_many_sequences_and_nan():
    g = H.gen(3)
    lens = torch.randint(0, 200, (1500,), generator=g).tolist()
    new = [int(torch.randint(0, n + 1, (1,), generator=g)) for n in lens]
    bt, pool = H.block_tables(g, lens, 16)
    kc = H.cache(g, pool, 2, 16, 64, F16)
    kc[bt[torch.tensor(lens).argmax(), 0], 1, 5, 7] = float("nan")
    kc[bt[torch.tensor(lens).argmax(), 1], 0, 5, 7] = float("-inf")
    kb = H.cache(g, pool, 2, 2, 64, F16)
    qsl = i32([0] + new).cumsum(0).to(torch.int32)
    assert_bounds(run_bounds(kb, kc, bt, i32(lens), qsl), kb, kc, bt, i32(lens), new)
    assert wllm.device_errors() == 0


@pytest.mark.parametrize("first", [1, 7, 40, 3000, 10 ** 9])
def test_bounds_of_chunks_behind_other_rows(first):
    """query_start_loc cut out of a batch's: its first entry is not zero (rows of other sequences come before)."""
    g = H.gen(first)
    lens, new = [64, 33, 0, 500], [64, 20, 0, 333]
    bt, pool = H.block_tables(g, lens, 16)
    kc, kb = H.cache(g, pool, 2, 16, 64, BF, bt, lens), H.cache(g, pool, 2, 2, 64, BF)
    qsl = (i32([0] + new).cumsum(0) + first).to(torch.int32)
    assert_bounds(run_bounds(kb, kc, bt, i32(lens), qsl), kb, kc, bt, i32(lens), new)
    assert wllm.device_errors() == 0


def test_bounds_of_forty_thousand_sequences():
    """More sequences than 16 bits count, as a decode may have; several name one block."""
    g = H.gen(15)
    B, pool = 40000, 700
    lens = torch.randint(0, 33, (B,), generator=g, dtype=torch.int32)
    bt = torch.randint(0, pool, (B, 4), generator=g, dtype=torch.int32)
    kc, kb = H.cache(g, pool, 2, 8, 64, BF), H.cache(g, pool, 2, 2, 64, BF)
    assert_bounds(run_bounds(kb, kc, bt, lens), kb, kc, bt, lens, (lens > 0).int())
    qsl = torch.cat([i32([0]), lens.cumsum(0).to(torch.int32)])
    assert_bounds(run_bounds(kb, kc, bt, lens, qsl), kb, kc, bt, lens, lens)
    assert wllm.device_errors() == 0


@pytest.mark.parametrize("starts", [[0, 32, 31, 90], [0, 40, 30, 31], [0, 100, 50, 200], [5, 4, 4, 4], [0, 64, 64, 63]])
def test_bounds_record_starts_that_decrease(starts):
    g = H.gen(14)
    lens = [320, 480, 640]
    bt, pool = H.block_tables(g, lens, 16)
    kc, kb = H.cache(g, pool, 1, 16, 64, BF), H.cache(g, pool, 1, 2, 64, BF)
    run_bounds(kb, kc, bt, i32(lens), i32(starts))
    assert wllm.device_errors() == 4


def test_bounds_record_bad_lengths_and_blocks(monkeypatch):
    g = H.gen(4)
    lens = [32, 48, 64]
    bt, pool = H.block_tables(g, lens, 16)
    kc, kb = H.cache(g, pool, 1, 16, 64, BF), H.cache(g, pool, 1, 2, 64, BF)
    bad = bt.clone()
    bad[1, 1] = pool
    got = run_bounds(kb, kc, bad, i32([32, 48, 9999]), i32([0, 32, 80, 144]))
    assert wllm.device_errors() == 2 | 4
    ref = S.key_bounds(kc, bt, i32([32, 48, 0]), [32, 48, 0], S.values(kb))
    ref[bt[1, 1]] = S.values(kb)[bt[1, 1]]
    assert torch.equal(S.values(got), ref)
    got = run_bounds(kb, kc, bt, i32(lens), i32([0, 40, 30, 31]))  # more new tokens than cached ones, a step back, one
    assert wllm.device_errors() == 4
    got = run_bounds(kb, kc, bt, i32(lens), i32([0, 0, 0, 10 ** 9]))  # more than the tables can name
    assert wllm.device_errors() == 4 and torch.equal(H.bits(got), H.bits(kb))
    monkeypatch.setenv("WLLM_CHECK", "1")
    with pytest.raises(wllm.WllmError, match="0x4"):
        run_bounds(kb, kc, bt, i32([32, 48, -1]))


# ---------------------------------------------------------------- selection
def run_select(q, kb, bt, cl, Hkv, bs, top, sink, recent):
    qd, kd, bd, cd = cuda(q, kb, bt, cl)
    sel = torch.full((q.shape[0], Hkv, top), -7, dtype=torch.int32, device="cuda")
    assert wllm.select_blocks(sel, qd, kd, bd, cd, Hkv, bs, sink, recent) is sel
    torch.cuda.synchronize()
    return sel.cpu()


def bounds_pool(g, pool, Hkv, D, dtype, spread=1.0):
    if dtype == U8:
        x = torch.randn(pool, Hkv, 2, D, generator=g) * 40
        return torch.stack([oracle.e4m3_encode(x.amin(2)), oracle.e4m3_encode(x.amax(2))], 2)
    x = H.randn(g, pool, Hkv, 2, D, scale=spread)
    return torch.stack([x.amin(2), x.amax(2)], 2).to(dtype)


def assert_selected(q, kb, bt, cl, Hkv, bs, top, sink, recent):
    got = run_select(q, kb, bt, cl, Hkv, bs, top, sink, recent)
    ref = S.select_blocks(q, kb, bt, cl, Hkv, bs, top, sink, recent)
    assert torch.equal(got, ref), (got != ref).nonzero()[:5]
    assert wllm.device_errors() == 0


@pytest.mark.parametrize("dtype,kind", [(F32, F32), (F16, F16), (BF, BF), (F16, U8), (BF, U8)])
@pytest.mark.parametrize("D,Hq,Hkv,bs,lens,top,sink,recent", [
    (128, 28, 4, 16, [1, 15, 16, 17, 300, 1000, 2500, 0], 20, 1, 2),
    (64, 8, 1, 8, [5000, 160, 161, 168, 169], 20, 0, 1),
    (256, 4, 4, 32, [4000, 4001], 3, 1, 1),
    (128, 32, 2, 64, [30000, 64 * 9 + 1], 9, 4, 5),      # no room for scored blocks
    (64, 6, 2, 256, [60000], 1, 0, 1),
    (128, 5, 5, 16, [70000], 130, 2, 9),
])
def test_selection_is_the_definitions(dtype, kind, D, Hq, Hkv, bs, lens, top, sink, recent):
    g = H.gen(D + Hq + top)
    bt, pool = H.block_tables(g, lens, bs)
    q = H.randn(g, len(lens), Hq, D, dtype=dtype)
    assert_selected(q, bounds_pool(g, pool, Hkv, D, kind), bt, i32(lens), Hkv, bs, top, sink, recent)


def test_selection_settles_equal_and_nearly_equal_scores():
    """Blocks that binary32 cannot tell apart: all alike, one of two values, and values 2^-9 apart on scores of 2^17."""
    g = H.gen(7)
    lens, bs, D = [16 * 1700, 16 * 90, 16 * 3000], 16, 64
    bt, pool = H.block_tables(g, lens, bs)
    q = torch.ones(3, 2, D, dtype=F32)
    kb = torch.ones(pool, 1, 2, D, dtype=F32)
    assert_selected(q, kb, bt, i32(lens), 1, bs, 40, 1, 2)
    kb[torch.randperm(pool, generator=g)[:pool // 2]] = 2.0
    assert_selected(q, kb, bt, i32(lens), 1, bs, 40, 1, 2)
    q = torch.ones(3, 2, D, dtype=BF)
    q[:, :, 0], q[:, :, 1] = 256.0, 2.0 ** -9
    kb = torch.zeros(pool, 1, 2, D, dtype=BF)
    kb[:, :, :, 0] = 256.0
    kb[:, :, :, 1] = torch.randint(0, 200, (pool, 1, 1), generator=g).to(BF)
    assert_selected(q, kb, bt, i32(lens), 1, bs, 40, 1, 2)
    kb[:, :, :, 0] = torch.randint(0, 3, (pool, 1, 1), generator=g).to(BF) * 128  # a few coarse levels besides
    assert_selected(q, kb, bt, i32(lens), 1, bs, 600, 1, 2)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
def test_selection_with_infinities_nan_and_extremes(dtype):
    g = H.gen(8)
    lens, bs, D = [16 * 300, 16 * 300, 16 * 300], 16, 128
    bt, pool = H.block_tables(g, lens, bs)
    q = H.randn(g, 3, 4, D, dtype=dtype)
    kb = bounds_pool(g, pool, 2, D, dtype)
    kb[bt[0, 17].long(), 0, 1, 3] = float("inf")
    kb[bt[0, 200].long(), 0, :, 5] = float("nan")
    kb[bt[0, 100].long(), 1, 0, 3] = -float("inf")
    big = torch.finfo(dtype).max
    kb[bt[1, 40:60].long(), :, 1, :] = big           # products that overflow binary32 for bf16 and f32
    q[1] = q[1].clamp(-1, 1) * (big if dtype != F16 else 1000.0)
    assert_selected(q, kb, bt, i32(lens), 2, bs, 33, 1, 3)
    q[2, 1, 7] = float("nan")
    assert_selected(q, kb, bt, i32(lens), 2, bs, 33, 1, 3)
    q[:] = 0
    assert_selected(q, bounds_pool(g, pool, 2, D, dtype, 1e-3), bt, i32(lens), 2, bs, 33, 1, 3)


def test_selection_strides_and_many_rows():
    g = H.gen(9)
    lens = torch.randint(1, 3000, (200,), generator=g).tolist()
    bt, pool = H.block_tables(g, lens, 16)
    kb = bounds_pool(g, pool, 3, 64, BF)
    wide = H.randn(g, 200, 9, 100, dtype=BF)
    sel = torch.full((200, 4, 50), -7, dtype=torch.int32, device="cuda")
    q, kd, bd, cd = cuda(wide, kb, bt, i32(lens))
    wllm.select_blocks(sel[:, :3, 1:31], q[:, 1:7, 3:67], kd, bd, cd, 3, 16, 2, 2)
    torch.cuda.synchronize()
    ref = S.select_blocks(wide[:, 1:7, 3:67].contiguous(), kb, bt, i32(lens), 3, 16, 30, 2, 2)
    assert torch.equal(sel[:, :3, 1:31].cpu(), ref)
    rest = sel.cpu()
    rest[:, :3, 1:31] = -7
    assert (rest == -7).all()


def test_selection_records_bad_tables_and_lengths(monkeypatch):
    g = H.gen(10)
    bt, pool = H.block_tables(g, [640, 640], 16)
    kb, q = bounds_pool(g, pool, 1, 64, F16), H.randn(g, 2, 2, 64, dtype=F16)
    bad = bt.clone()
    bad[0, 5] = -1
    run_select(q, kb, bad, i32([640, 640]), 1, 16, 8, 1, 1)
    assert wllm.device_errors() == 2
    run_select(q, kb, bt, i32([640, 9999]), 1, 16, 8, 1, 1)
    assert wllm.device_errors() == 4
    monkeypatch.setenv("WLLM_CHECK", "1")
    with pytest.raises(wllm.WllmError, match="0x4"):
        run_select(q, kb, bt, i32([640, -3]), 1, 16, 8, 1, 1)


# ---------------------------------------------------------------- sparse decode
KS, VS = 0.03125, 0.02


def run_sparse(q, kc, vc, bt, cl, sel, scale, out=None):
    qd, kd, vd, bd, cd, sd = cuda(q, kc, vc, bt, cl, sel)
    o = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda") if out is None else out
    bs, Hkv = kc.shape[2], kc.shape[1]
    if kc.dtype == U8:
        got = wllm.paged_attention_decode_sparse_fp8(o, qd, kd, vd, bd, cd, sd, Hkv, scale, KS, VS, bs)
    else:
        got = wllm.paged_attention_decode_sparse(o, qd, kd, vd, bd, cd, sd, Hkv, scale, bs)
    assert got is o
    torch.cuda.synchronize()
    return o.cpu()


def sparse_ref(q, kc, vc, bt, cl, sel, scale):
    fp8 = kc.dtype == U8
    return S.sparse_decode(q, kc, vc, bt, cl, sel, float(torch.tensor(scale, dtype=F32)), KS if fp8 else 1.0, VS if fp8 else 1.0)


def lists(g, lens, Hkv, bs, top, ordered=True):
    """Random selections of every row's blocks: as many as there are or fit, some rows with fewer, some with gaps."""
    sel = torch.full((len(lens), Hkv, top), -1, dtype=torch.int32)
    for b, L in enumerate(lens):
        n = -(-L // bs)
        for h in range(Hkv):
            count = min(n, top) if (b + h) % 3 else int(torch.randint(0, min(n, top) + 1, (1,), generator=g))
            ids = torch.randperm(n, generator=g)[:count]
            if n and count and (b + h) % 2:
                ids[0] = n - 1 if n - 1 not in ids[1:].tolist() else ids[0]
            if ordered:
                sel[b, h, :count] = ids.sort().values.to(torch.int32)
            else:
                sel[b, h, torch.randperm(top, generator=g)[:count]] = ids.to(torch.int32)
    return sel


@pytest.mark.parametrize("dtype,kind", [(F32, F32), (F16, F16), (BF, BF), (F16, U8), (BF, U8)])
@pytest.mark.parametrize("D,Hq,Hkv,bs,lens,top", [
    (128, 28, 4, 16, [1, 16, 17, 333, 2000, 0, 40], 12),
    (64, 8, 8, 8, [5, 900, 64, 77, 1], 33),
    (64, 32, 4, 16, [700, 30], 40),
    (128, 32, 2, 32, [1000, 33, 64, 5], 9),          # 16 query heads a kv head
    (256, 8, 1, 16, [3000, 250, 1], 70),
    (128, 20, 1, 64, [900, 64, 63], 5),              # 20: two tiles, the second short
    (256, 5, 1, 256, [2000, 300], 4),
    (128, 8, 8, 16, [4000], 250),
    (64, 3, 3, 128, [1], 1),
])
def test_sparse_decode_matches_binary64(dtype, kind, D, Hq, Hkv, bs, lens, top):
    g = H.gen(D + Hq + bs + top)
    bt, pool = H.block_tables(g, lens, bs)
    kc, vc = (H.cache(g, pool, Hkv, bs, D, kind, bt, lens) for _ in range(2))
    q = H.randn(g, len(lens), Hq, D, dtype=dtype)
    if kind == U8 and D == 64 and bs < 16:  # as for every call over an fp8 cache
        with pytest.raises(wllm.WllmError, match="block_size >= 16"):
            run_sparse(q, kc, vc, bt, i32(lens), lists(g, lens, Hkv, bs, top), 0.1)
        return
    for ordered in (True, False):
        sel = lists(g, lens, Hkv, bs, top, ordered)
        got = run_sparse(q, kc, vc, bt, i32(lens), sel, 1 / math.sqrt(D))
        ref, mag, size = sparse_ref(q, kc, vc, bt, i32(lens), sel, 1 / math.sqrt(D))
        H.assert_sparse(got, ref, mag, size, dtype, kind == U8, f"ordered {ordered}")
        empty = mag.sum(-1) == 0
        assert (got[empty] == 0).all()
    assert wllm.device_errors() == 0


@pytest.mark.parametrize("dtype,kind", [(F16, F16), (BF, BF), (F16, U8), (BF, U8)])
@pytest.mark.parametrize("Hq,Hkv,bs", [(8, 1, 16), (32, 2, 16), (5, 5, 32)])
def test_sparse_decode_keeps_its_weights(dtype, kind, Hq, Hkv, bs):
    """The softmax weights are not rounded to 16 bits on their way to the output.

    Scores are small and lists hold 64 tokens at most, so everything but the output's own rounding is small.  A score is off
    by at most size * (4 products of 16 terms, each instruction within 17 * 2^-22 of the magnitudes in it, = 272 * 2^-24,
    and 8 roundings of scaling and difference), where size = max scale sum |q k|; its exponential by 2^-21 more; both
    count twice (numerator and sum).  Two words of bf16, the first one cut off, leave off 2^-7 * 2^-8 of a weight, two of f16
    2^-10 * 2^-11 or, at the subnormal end, 2^-25 of the largest, 1: with weights above 1/16 (scores within 4 log2 units) n
    of those over their sum are at most 2^-21.  The products with v are up to 8 instructions, 17 * 2^-22 each, and merging and
    scaling 16 roundings.  One word would leave off 2^-9 or 2^-12 of a weight: several times this bound."""
    g = H.gen(Hq + bs)
    D, B, scale = 64, 48, 0.0125
    lens = [64] * B
    bt, pool = H.block_tables(g, lens, bs)
    kc, vc = (H.cache(g, pool, Hkv, bs, D, kind, bt, lens) for _ in range(2))
    q = H.randn(g, B, Hq, D, dtype=dtype)
    q = torch.where(q.abs() < 2.0 ** -13, torch.ones_like(q), q)  # exact as f16 also from bf16
    sel = torch.arange(64 // bs, dtype=torch.int32).expand(B, Hkv, -1).contiguous()
    got = run_sparse(q, kc, vc, bt, i32(lens), sel, scale)
    ref, mag, size = sparse_ref(q, kc, vc, bt, i32(lens), sel, scale)
    assert 2 * size.max() * math.log2(math.e) < 4
    word = 2.0 ** -15 if dtype == BF and kind != U8 else 2.0 ** -21
    d = 2 * (torch.expm1(size * 280 * H.U32)[..., None] + 2.0 ** -21) + word + 8 * 17 * 2.0 ** -22 + 16 * H.U32
    vmax = S.values(vc).nan_to_num(0.0).abs().max() * (VS if kind == U8 else 1.0)
    tol = d * mag + 2.0 ** -21 * vmax + H.HALF[dtype] * ref.abs() + H.TINY[dtype]
    off = (got.double() - ref).abs()
    assert (off <= tol).all(), f"{int((off > tol).sum())} off, worst {(off / tol).max().item():.2f} of its bound"


@pytest.mark.parametrize("kind", [F32, BF, F16])
@pytest.mark.parametrize("D,Hq,top", [(64, 4, 3), (128, 9, 40), (256, 2, 40)])
def test_sparse_decode_of_infinite_values(kind, D, Hq, top):
    """A value of +-inf with a positive weight comes out infinite, both signs or NaN as NaN, and other elements are as ever;
    on a row's last token and behind it, where the value is NaN and not looked at."""
    g = H.gen(D)
    lens = [700, 33, 17]
    bt, pool = H.block_tables(g, lens, 16)
    kc, vc = (H.cache(g, pool, 1, 16, D, kind, bt, lens) for _ in range(2))
    inf = float("inf")
    for b, n in enumerate(lens):
        at = lambda t: (int(bt[b, t // 16]), 0, t % 16)  # noqa: E731
        vc[at(n - 1)][1], vc[at(0)][2], vc[at(1)][2] = inf, -inf, -inf
        vc[at(0)][3], vc[at(n - 1)][3], vc[at(2)][5] = inf, -inf, float("nan")
        for t in range(16):
            vc[at(t)][D - 1] = inf
    q = H.randn(g, 3, Hq, D, dtype=kind)
    sel = torch.full((3, 1, top), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        last = (n - 1) // 16
        sel[b, 0, :2] = i32([0, last])
        sel[b, 0, 2:2 + min(top - 2, max(0, last - 1))] = torch.arange(1, last, dtype=torch.int32)[:top - 2]
    got = run_sparse(q, kc, vc, bt, i32(lens), sel, 0.02)
    ref, mag, size = sparse_ref(q, kc, vc, bt, i32(lens), sel, 0.02)
    want = {1: inf, 2: -inf, D - 1: inf}
    for i, x in want.items():
        assert (ref[..., i] == x).all() and (got[..., i] == x).all(), i
    for i in (3, 5):
        assert ref[..., i].isnan().all() and got[..., i].isnan().all(), i
    rest = [i for i in range(D) if i not in (1, 2, 3, 5, D - 1)]
    H.assert_sparse(got[..., rest], ref[..., rest], mag[..., rest], size, kind, False, "beside infinities")


@pytest.mark.parametrize("kind", [F32, BF, U8])
def test_sparse_decode_of_every_block_is_the_decode(kind):
    g = H.gen(20)
    lens = [1, 100, 257, 1500]
    dtype = F16 if kind == U8 else kind
    bt, pool = H.block_tables(g, lens, 16)
    kc, vc = (H.cache(g, pool, 4, 16, 128, kind, bt, lens) for _ in range(2))
    q = H.randn(g, 4, 28, 128, dtype=dtype)
    sel = torch.arange(bt.shape[1], dtype=torch.int32).expand(4, 4, -1)
    sel = torch.where(sel < ((i32(lens) + 15) // 16)[:, None, None], sel, -1).contiguous()
    got = run_sparse(q, kc, vc, bt, i32(lens), sel, 0.1)
    qd, kd, vd, bd, cd = cuda(q, kc, vc, bt, i32(lens))
    out = torch.empty_like(qd)
    if kind == U8:
        wllm.paged_attention_decode_fp8(out, qd, kd, vd, bd, cd, 4, 0.1, KS, VS, 16)
    else:
        wllm.paged_attention_decode(out, qd, kd, vd, bd, cd, 4, 0.1, 16)
    ref, mag, size = sparse_ref(q, kc, vc, bt, i32(lens), sel, 0.1)
    H.assert_sparse(got, ref, mag, size, dtype, kind == U8, "sparse")
    H.assert_sparse(out.cpu(), ref, mag, size, dtype, kind == U8, "decode")


def test_sparse_decode_strides_negative_scale_and_large_scores():
    g = H.gen(21)
    lens = [500, 90]
    bt, pool = H.block_tables(g, lens, 16)
    kc, vc = (H.cache(g, pool, 2, 16, 64, F16, bt, lens) for _ in range(2))
    wide_q, wide_o = H.randn(g, 2, 7, 80, dtype=F16), torch.full((2, 9, 70), 3.0, dtype=F16, device="cuda")
    sel = lists(g, lens, 2, 16, 11)
    wide_s = torch.full((2, 3, 14), 5, dtype=torch.int32)
    wide_s[:, 1:, 2:13] = sel
    q = wide_q[:, 1:5, 5:69]
    qd, sd = wide_q.cuda()[:, 1:5, 5:69], wide_s.cuda()[:, 1:, 2:13]
    kd, vd, bd, cd = cuda(kc, vc, bt, i32(lens))
    wllm.paged_attention_decode_sparse(wide_o[:, 2:6, 3:67], qd, kd, vd, bd, cd, sd, 2, -0.3, 16)
    torch.cuda.synchronize()
    ref, mag, size = sparse_ref(q.contiguous(), kc, vc, bt, i32(lens), sel, -0.3)
    H.assert_sparse(wide_o[:, 2:6, 3:67].cpu(), ref, mag, size, F16, False, "strided")
    rest = wide_o.cpu()
    rest[:, 2:6, 3:67] = 3.0
    assert (rest == 3.0).all()
    q = H.randn(g, 2, 4, 64, dtype=F16, scale=30.0)
    got = run_sparse(q, kc, vc, bt, i32(lens), sel, 1.0)
    ref, mag, size = sparse_ref(q, kc, vc, bt, i32(lens), sel, 1.0)
    H.assert_sparse(got, ref, mag, size, F16, False, "large scores")


def test_sparse_decode_lists_a_block_twice_and_records_bad_entries(monkeypatch):
    g = H.gen(22)
    lens = [100, 100]
    bt, pool = H.block_tables(g, lens, 16)
    kc, vc = (H.cache(g, pool, 1, 16, 64, BF, bt, lens) for _ in range(2))
    q = H.randn(g, 2, 4, 64, dtype=BF)
    sel = i32([[[3, 1, 3]], [[6, -1, 6]]])
    got = run_sparse(q, kc, vc, bt, i32(lens), sel, 0.125)
    ref, mag, size = sparse_ref(q, kc, vc, bt, i32(lens), sel, 0.125)
    H.assert_sparse(got, ref, mag, size, BF, False, "twice")
    bad = i32([[[3, 7, 1]], [[2, 2000000000, -5]]])
    got = run_sparse(q, kc, vc, bt, i32(lens), bad, 0.125)
    assert wllm.device_errors() == 2
    good = i32([[[3, -1, 1]], [[2, -1, -1]]])
    ref, mag, size = sparse_ref(q, kc, vc, bt, i32(lens), good, 0.125)
    H.assert_sparse(got, ref, mag, size, BF, False, "bad entries")
    table = bt.clone()
    table[0, 3] = pool
    run_sparse(q, kc, vc, table, i32(lens), good, 0.125)
    assert wllm.device_errors() == 2
    run_sparse(q, kc, vc, bt, i32([100, 5000]), good, 0.125)
    assert wllm.device_errors() == 4
    monkeypatch.setenv("WLLM_CHECK", "1")
    with pytest.raises(wllm.WllmError, match="0x2"):
        run_sparse(q, kc, vc, bt, i32(lens), bad, 0.125)


# ---------------------------------------------------------------- together
class Layer:
    """One layer's caches and the four calls of a step over them."""

    def __init__(self, seed, lens, room, Hq=8, Hkv=2, D=128, bs=16, dtype=BF, fp8=False, top=6, sink=1, recent=2):
        g = H.gen(seed)
        self.g, self.lens, self.bs, self.dtype, self.fp8 = g, list(lens), bs, dtype, fp8
        self.Hq, self.Hkv, self.D, self.top, self.sink, self.recent = Hq, Hkv, D, top, sink, recent
        kind = U8 if fp8 else dtype
        self.bt, pool = H.block_tables(g, [n + room for n in lens], bs)
        self.kc, self.vc = (H.cache(g, pool, Hkv, bs, D, kind).cuda() for _ in range(2))
        self.kb = H.cache(g, pool, Hkv, 2, D, kind).cuda()
        self.table, self.weight = H.rotary_table(4096, D).cuda(), (1 + H.randn(g, D, scale=0.2)).to(dtype).cuda()
        self.btd = self.bt.cuda()
        self.scale = 1 / math.sqrt(D)

    def tokens(self, counts):
        """New tokens of every sequence behind what it holds: fused rows, slots and positions; lens grow."""
        pos = torch.cat([torch.arange(n, n + c) for n, c in zip(self.lens, counts)])
        seq = torch.arange(len(counts)).repeat_interleave(torch.tensor(counts))
        slots = self.bt[seq, pos // self.bs].long() * self.bs + pos % self.bs
        fused = H.randn(self.g, len(pos), (self.Hq + 2 * self.Hkv) * self.D, dtype=self.dtype)
        self.lens = [n + c for n, c in zip(self.lens, counts)]
        return [x.cuda() for x in (fused, slots, pos, i32(self.lens), i32([0] + list(counts)).cumsum(0).to(torch.int32))]

    def append(self, fused, slots, pos):
        T, D = fused.shape[0], self.D
        q, k, v = (fused[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, self.Hq), (self.Hq, self.Hq + self.Hkv), (self.Hq + self.Hkv, self.Hq + 2 * self.Hkv)))
        how = dict(q_weight=self.weight, k_weight=self.weight)
        if self.fp8:
            return wllm.rotate_and_cache_fp8(q, q, k, v, self.kc, self.vc, slots, pos, self.table, KS, VS, **how)
        return wllm.rotate_and_cache(q, q, k, v, self.kc, self.vc, slots, pos, self.table, **how)

    def attend(self, q, cl, sel, out):
        wllm.update_key_bounds(self.kb, self.kc, self.btd, cl, self.bs)
        wllm.select_blocks(sel, q, self.kb, self.btd, cl, self.Hkv, self.bs, self.sink, self.recent)
        args = (out, q, self.kc, self.vc, self.btd, cl, sel, self.Hkv, self.scale)
        if self.fp8:
            return wllm.paged_attention_decode_sparse_fp8(*args, KS, VS, self.bs)
        return wllm.paged_attention_decode_sparse(*args, self.bs)

    def new(self):
        B = len(self.lens)
        return (torch.empty(B, self.Hkv, self.top, dtype=torch.int32, device="cuda"),
                torch.empty(B, self.Hq, self.D, dtype=self.dtype, device="cuda"))

    def check(self, q, cl, sel, out, what):
        """What the calls left, against the definitions on the caches as they are."""
        kc, vc, kb, q, cl = (x.cpu() for x in (self.kc, self.vc, self.kb, q, cl))
        full = S.key_bounds(kc, self.bt, cl, cl, S.values(kb))
        for b, n in enumerate(cl.tolist()):
            ids = self.bt[b, :n // self.bs].long()
            assert torch.equal(S.values(kb)[ids], full[ids]), f"{what}: bounds of {b}"
        ref = S.select_blocks(q.contiguous(), kb, self.bt, cl, self.Hkv, self.bs, self.top, self.sink, self.recent)
        assert torch.equal(sel.cpu(), ref), f"{what}: selection"
        H.assert_sparse(out.cpu(), *sparse_ref(q.contiguous(), kc, vc, self.bt, cl, ref, self.scale), self.dtype, self.fp8, what)


@pytest.mark.parametrize("dtype,fp8", [(BF, False), (F16, True), (F32, False)])
def test_prompt_and_steps(dtype, fp8):
    layer = Layer(30, [0, 0, 0], 260, dtype=dtype, fp8=fp8)
    fused, slots, pos, cl, qsl = layer.tokens([200, 31, 77])
    layer.append(fused, slots, pos)
    wllm.update_key_bounds(layer.kb, layer.kc, layer.btd, cl, layer.bs, query_start_loc=qsl)
    for step in range(20):
        fused, slots, pos, cl, _ = layer.tokens([1, 1, 1])
        q = layer.append(fused, slots, pos)
        sel, out = layer.new()
        layer.attend(q, cl, sel, out)
        torch.cuda.synchronize()
        layer.check(q, cl, sel, out, f"step {step}")
    assert wllm.device_errors() == 0


def test_captured_step_replayed_with_new_inputs():
    """A step captured once and replayed on other inputs and lengths, a second captured graph on its own tensors in
    between, and eager calls on another stream meanwhile."""
    a, b = Layer(31, [150, 0, 333], 100), Layer(32, [40, 700], 100, Hkv=1, top=9)
    graphs = []
    for layer in (a, b):
        fused, slots, pos, cl, qsl = layer.tokens([20] * len(layer.lens))
        layer.append(fused, slots, pos)
        wllm.update_key_bounds(layer.kb, layer.kc, layer.btd, cl, layer.bs, query_start_loc=cl.new_tensor([0] + layer.lens).cumsum(0).to(torch.int32))
        static = layer.tokens([1] * len(layer.lens))[:4]
        sel, out = layer.new()
        q = layer.append(*static[:3])
        layer.attend(q, static[3], sel, out)  # the first call of each kernel is not captured
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q = layer.append(*static[:3])
            layer.attend(q, static[3], sel, out)
        graphs.append((layer, graph, static, q, sel, out))
    other = Layer(33, [500, 90], 20)
    side = torch.cuda.Stream()
    for step in range(18):
        for layer, graph, static, q, sel, out in graphs:
            for s, x in zip(static, layer.tokens([1] * len(layer.lens))):
                s.copy_(x)
            graph.replay()
        fresh = other.tokens([1, 1]) if step == 0 else fresh
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            oq = other.append(fresh[0].clone(), *fresh[1:3])
            osel, oout = other.new()
            other.attend(oq, fresh[3], osel, oout)
        torch.cuda.synchronize()
        for layer, graph, static, q, sel, out in graphs:
            layer.check(q, static[3], sel, out, f"replay {step}")
        if step == 0:
            want = oout.clone(), osel.clone()
            ref = sparse_ref(oq.cpu().contiguous(), other.kc.cpu(), other.vc.cpu(), other.bt, fresh[3].cpu(), osel.cpu(), other.scale)
            H.assert_sparse(oout.cpu(), *ref, BF, False, "other stream")
        assert torch.equal(oout, want[0]) and torch.equal(osel, want[1])  # the same inputs, the same bits
    assert wllm.device_errors() == 0


def test_threads_call_at_once():
    """Steps of four layers, each in a thread and on a stream of its own, with tables of several widths (the selection's
    shared memory grows with them), give the bits that they give one after another."""
    def step(layer, inputs):
        fused, slots, pos, cl = inputs
        q = layer.append(fused.clone(), slots, pos)
        sel, out = layer.new()
        layer.attend(q, cl, sel, out)
        return q.clone(), sel, out

    layers = [Layer(40 + i, lens, extra) for i, (lens, extra) in enumerate(
        [([150, 333], 40), ([900], 3000), ([64, 1200, 31], 9000), ([2000], 20000)])]
    work = []
    for layer in layers:
        n = len(layer.lens)
        fused, slots, pos, cl, qsl = layer.tokens([40] * n)
        layer.append(fused, slots, pos)
        wllm.update_key_bounds(layer.kb, layer.kc, layer.btd, cl, layer.bs,
                               query_start_loc=cl.new_tensor([0] + layer.lens).cumsum(0).to(torch.int32))
        inputs = layer.tokens([1] * n)[:4]
        work.append((layer, inputs, step(layer, inputs)))
    torch.cuda.synchronize()
    got = [None] * len(work)

    def run(i):
        layer, inputs, _ = work[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got[i] = step(layer, inputs)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for (layer, inputs, want), have in zip(work, got):
        assert all(torch.equal(x, y) for x, y in zip(want, have)), "a thread's step"
    assert wllm.device_errors() == 0
