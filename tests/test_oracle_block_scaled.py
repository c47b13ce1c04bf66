"""The definitions of the block-scaled cache's calls against brute force, closed forms and the per-tensor ones."""
import math

import pytest
import torch

import oracle
from oracle import block_scaled as S
from oracle import sparse
from tests import block_scaled_helpers as K
from tests import sparse_helpers as H

BF, I32 = torch.bfloat16, torch.int32


@pytest.mark.parametrize("m,e", [(448.0, 0), (448.0 * (1 + 2 ** -23), 1), (1.0, -8), (1.75, -8), (1.7500001, -7), (0.0, -40),
                                 (2.0 ** -60, -40), (3e38, 40), (448 * 2.0 ** 40, 40), (1e-30, -40)])
def test_scale_is_the_least_power_of_two(m, e):
    x = torch.tensor([[0.5 * m, -m, math.inf, math.nan, 0.0]], dtype=torch.float32)
    assert S.block_scale(x) == 2.0 ** e
    if -40 < e < 40:
        assert m <= 448 * 2.0 ** e and m > 448 * 2.0 ** (e - 1)


def test_fresh_blocks_are_the_per_tensor_append_with_their_scale():
    g, bs, hkv, d = H.gen(1), 8, 2, 32
    key, value = H.randn(g, 20, hkv, d, dtype=BF), H.randn(g, 20, hkv, d, dtype=BF, scale=9.0)
    caches = [torch.zeros(4, hkv, bs, d, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.full((4, hkv), math.nan) for _ in range(2)]
    S.append(key, value, *caches, *scales, torch.tensor([[2, 0, 3]], dtype=I32), torch.tensor([20], dtype=I32), torch.tensor([0, 20], dtype=I32))
    for x, c, s in zip((key, value), caches, scales):
        assert s[1].isnan().all() and not c[1].any()
        for h in range(hkv):
            for j, block in enumerate((2, 0, 3)):
                rows = x[j * bs:(j + 1) * bs, h].float()
                k = math.frexp(rows.abs().max().item() / 448)
                assert s[block, h].item() == 2.0 ** (k[1] if k[0] > 0.5 else k[1] - 1)
                ref = (rows / s[block, h]).to(torch.float8_e4m3fn)
                assert torch.equal(c[block, h, :rows.shape[0]], ref.view(torch.uint8))


def test_a_rise_stores_the_earlier_codes_again():
    d, bs = 16, 8
    caches = [torch.full((1, 1, bs, d), 0x7f, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.full((1, 1), math.nan) for _ in range(2)]
    table, x = torch.tensor([[0]], dtype=I32), torch.zeros(1, 1, d)
    x[0, 0, :4] = torch.tensor([448.0, 2.0 ** -6, 3 * 2.0 ** -9, -1.0])
    S.append(x, x, *caches, *scales, table, torch.tensor([1], dtype=I32))
    assert scales[0].item() == 1.0
    S.append(x * 2, x, *caches, *scales, table, torch.tensor([2], dtype=I32))
    assert scales[0].item() == 2.0 and scales[1].item() == 1.0
    got = oracle.widen_e4m3(caches[0][0, 0])
    assert got[0, :4].tolist() == [224.0, 2.0 ** -7, 2 * 2.0 ** -9, -0.5]  # 1.5 2^-9 went to the even code
    assert got[1, :4].tolist() == [448.0, 2.0 ** -6, 3 * 2.0 ** -9, -1.0] and got[2:].isnan().all()
    S.append(x / 4, x, *caches, *scales, table, torch.tensor([3], dtype=I32))    # a smaller token changes nothing
    assert scales[0].item() == 2.0 and torch.equal(oracle.widen_e4m3(caches[0][0, 0, :2]), got[:2])
    S.append(x / 4, x, *caches, *scales, table, torch.tensor([1], dtype=I32))    # the first token again: a new start
    assert scales[0].item() == 0.25


def test_attention_is_the_dense_one_on_what_codes_stand_for():
    g, lens = H.gen(2), [5, 1, 0, 33]
    bt, blocks = H.block_tables(g, lens, 8)
    kc, ks = K.pool(g, blocks, 2, 8, 64, bt, lens)
    vc, vs = K.pool(g, blocks, 2, 8, 64, bt, lens)
    q = H.randn(g, 4, 6, 64, dtype=BF)
    out, mag, size, least = S.attention(q, kc, vc, ks, vs, bt, torch.tensor(lens, dtype=I32), 0.2)
    assert not out[2].any()
    for b, n in enumerate(lens):
        at = [(int(bt[b, t // 8]), t % 8) for t in range(n)]
        for h in range(6) if n else ():
            k = torch.stack([oracle.widen_e4m3(kc[i, h // 3, o]) * ks[i, h // 3].double() for i, o in at])
            v = torch.stack([oracle.widen_e4m3(vc[i, h // 3, o]) * vs[i, h // 3].double() for i, o in at])
            p = torch.softmax(k @ q[b, h].double() * 0.2, 0)
            assert torch.allclose(out[b, h], p @ v, rtol=1e-12, atol=1e-15)
            assert torch.allclose(mag[b, h], p @ v.abs(), rtol=1e-12) and least[b, h] == n * max(vs[i, h // 3].item() for i, _ in at)
    # with one scale everywhere it is the fp8 decode
    one = torch.full_like(ks, 0.25)
    same, _, _ = sparse.sparse_decode(q, kc, vc, bt, torch.tensor(lens), torch.arange(5).expand(4, 2, 5), 0.2, 0.25, 0.25)
    assert torch.allclose(S.attention(q, kc, vc, one, one, bt, torch.tensor(lens), 0.2)[0], same, rtol=1e-12)


def test_chunks_are_rows_of_the_decode():
    g, lens, new = H.gen(3), [20, 9], [7, 9]
    bt, blocks = H.block_tables(g, lens, 8)
    kc, ks = K.pool(g, blocks, 1, 8, 64, bt, lens)
    q, starts = H.randn(g, 16, 2, 64), torch.tensor([0, 7, 16], dtype=I32)
    out = S.attention(q, kc, kc, ks, ks, bt, torch.tensor(lens), 0.2, starts)[0]
    for b in range(2):
        for i in range(new[b]):
            one = S.attention(q[starts[b] + i][None], kc, kc, ks, ks, bt[b:b + 1], torch.tensor([lens[b] - new[b] + i + 1]), 0.2)[0]
            assert torch.allclose(out[starts[b] + i], one[0], rtol=1e-12)


def test_slots_by_hand():
    table = torch.tensor([[7, 8, -1], [9, -1, -1], [3, 4, -1], [-1, -1, -1]], dtype=I32)
    stack = torch.tensor([11, 12, 13, -1, -1, -1], dtype=I32)
    slots, pos, starts, lens, count, tab, st = S.assign_slots(
        table, torch.tensor([5, 3, 6, 0]), torch.tensor([4, 1, -1, 2]), stack, 3, 8, 4)
    assert lens.tolist() == [9, 4, 0, 2] and starts.tolist() == [0, 4, 5, 5, 7]
    assert st.tolist() == [11, 12, 13, 3, 4, -1] and count == 3
    assert tab[0].tolist() == [7, 8, 4] and tab[3].tolist() == [3, -1, -1]
    assert slots.tolist() == [33, 34, 35, 16, 39, 12, 13, -1] and pos.tolist() == [5, 6, 7, 8, 3, 0, 1, 0]


def test_slots_when_rows_or_blocks_run_short():
    table = torch.full((3, 4), -1, dtype=I32)
    stack = torch.tensor([5, 6], dtype=I32)
    call = lambda lens, new, rows, n=2: S.assign_slots(table, torch.tensor(lens), torch.tensor(new), stack, n, rows, 4)  # noqa: E731
    assert call([0, 0, 0], [4, 8, 4], 20)[2].tolist() == [0, 4, 4, 4]    # the second needs more than is left: no later one gets any
    table[2, 0] = 9
    assert call([0, 0, 1], [4, 8, 2], 20)[2].tolist() == [0, 4, 4, 6]    # but one that needs none is served
    assert call([0, 0, 0], [4, 4, 1], 7)[2].tolist() == [0, 4, 4, 4]     # rows: the same order
    assert call([0, 0, 0], [4, 17, 4], 20)[2].tolist() == [0, 4, 4, 8]   # too long for its table: counts for neither sum
