"""Slot assignment where rows that are given back hold entries that name no block: they do not get onto the stack."""
import pytest
import torch

import paged_kv_cache_185_gb300 as wllm
from oracle import block_scaled as S
from tests import sparse_helpers as H
from tests.test_gpu_block_scaled import assign, i32, slot_inputs

pytestmark = pytest.mark.gpu
NAMES = ("slots", "positions", "starts", "lengths", "count", "tables")
BLOCK = 2  # the bit of the error word


def check(table, lens, new, stack, count, rows, bs, in_place=True, err=BLOCK):
    assert wllm.device_errors() == 0
    got = assign(table, lens, new, stack, count, rows, bs, in_place=in_place)
    assert wllm.device_errors() == err
    ref = S.assign_slots(table, lens, new, stack, count, rows, bs)
    for name, a, b in zip(NAMES, got, ref):
        assert torch.equal(a.view(-1), b.view(-1) if torch.is_tensor(b) else i32([b])), name
    left = int(got[4])
    assert torch.equal(got[6][:left], ref[6][:left]) and (got[6][:left] >= 0).all()
    return got


def test_a_negative_entry_is_lost_and_harms_nobody():
    table = i32([[7, -1, 9], [3, -1, -1], [-1, -1, -1]])
    stack = i32([20, -9, -9, -9, -9])
    got = check(table, i32([10, 3, 0]), i32([-1, 2, 8]), stack, 1, 16, 4)
    # 7 and 9 came back on top of 20; sequence 1 takes 9, sequence 2 takes 7 and 20
    assert got[5].tolist() == [[7, -1, 9], [3, 9, -1], [7, 20, -1]] and int(got[4]) == 0
    assert got[0][:10].tolist() == [15, 36, 28, 29, 30, 31, 80, 81, 82, 83]
    # step after step: the pool holds what it held before
    again = check(got[5], got[3], i32([1, -1, -1]), torch.cat([got[6]]), int(got[4]), 4, 4, err=0)
    assert sorted(again[6][:int(again[4])].tolist() + [int(again[5][0, 0])]) == [3, 7, 9, 20]


def test_who_is_served_goes_by_the_blocks_that_there_are():
    """One block fewer than lengths say: the last sequence is not served, and stays as it was."""
    table = i32([[5, -2 ** 31], [-1, -1], [-1, -1]])
    got = check(table, i32([8, 0, 0]), i32([-1, 4, 4]), i32([-9] * 3), 0, 16, 4)
    assert got[3].tolist() == [0, 4, 0] and got[2].tolist() == [0, 0, 4, 4] and int(got[4]) == 0


@pytest.mark.parametrize("B,hi,most_new,bs,rows", [(3, 200, 40, 8, 100), (33, 64, 20, 32, 700), (300, 900, 300, 8, 40000),
                                                  (1025, 50, 5, 16, 4000), (16384, 9, 2, 16, 20000)])
@pytest.mark.parametrize("share", [0.02, 0.5, 1.0])
@pytest.mark.parametrize("in_place", [True, False])
def test_many(B, hi, most_new, bs, rows, share, in_place):
    table, lens, new, stack, count = slot_inputs(B + hi, B, hi, most_new, bs, ended=0.4, spare=B // 2, room=1 << 16)
    new[0], lens[0] = -1, hi
    g = H.gen(B)
    gone = (new < 0)[:, None] & (torch.rand(table.shape, generator=g) < share)
    gone[0, 0] = True
    table = torch.where(gone, torch.full_like(table, -1), table)
    table[0, 0] = -2 ** 31
    check(table, lens, new, stack, count, rows, bs, in_place=in_place)


def test_captured_and_replayed():
    """What a call leaves behind serves the next replay."""
    table, lens = i32([[7, -1, 9], [3, -1, -1], [-1, -1, -1]]).cuda(), i32([10, 3, 0]).cuda()
    stack, count, new = i32([20, -9, -9, -9, -9]).cuda(), i32([1]).cuda(), torch.zeros(3, dtype=torch.int32, device="cuda")
    slots, starts = torch.empty(16, dtype=torch.int64, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    wllm.assign_slots(slots, starts, table, lens, new, stack, count, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wllm.assign_slots(slots, starts, table, lens, new, stack, count, 4)
    held = [x.cpu() for x in (table, lens, stack, count)]
    for step, err in ((i32([-1, 2, 8]), BLOCK), (i32([3, 1, -1]), 0), (i32([-1, -1, 2]), 0)):
        new.copy_(step)
        graph.replay()
        torch.cuda.synchronize()
        ref = S.assign_slots(held[0], held[1], step, held[2], int(held[3]), 16, 4)
        assert wllm.device_errors() == err
        assert torch.equal(slots.cpu(), ref[0]) and torch.equal(lens.cpu(), ref[3]) and int(count) == ref[4] and torch.equal(table.cpu(), ref[5])
        held = [x.cpu() for x in (table, lens, stack, count)]
