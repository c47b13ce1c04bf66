"""Forms of block selection and block-sparse decode that only large calls take: batches beyond one wave of clusters, lists
of more units than a warp looks up at once, rows started longest first, the widest tables, and first launches that race."""
import os
import subprocess
import sys

import pytest
import torch

import paged_kv_cache_185_gb300 as wllm
from oracle import sparse as S
from tests import sparse_helpers as H
from tests.test_gpu_sparse import BF, F16, F32, U8, assert_selected, bounds_pool, i32, lists, run_sparse, sparse_ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def shared_pool(g, lens, bs, pool):
    """Tables whose entries are any blocks of a small pool, so that many sequences need little memory."""
    width = max(-(-n // bs) for n in lens)
    return torch.randint(0, pool, (len(lens), width), generator=g, dtype=torch.int32)


def check_sparse(dtype, kind, D, Hq, Hkv, bs, lens, top, seed):
    g = H.gen(seed)
    pool = 150
    bt = shared_pool(g, lens, bs, pool)
    kc, vc = (H.cache(g, pool, Hkv, bs, D, kind) for _ in range(2))
    q = H.randn(g, len(lens), Hq, D, dtype=dtype)
    sel = lists(g, lens, Hkv, bs, top)
    got = run_sparse(q, kc, vc, bt, i32(lens), sel, D ** -0.5)
    ref, mag, size = sparse_ref(q, kc, vc, bt, i32(lens), sel, D ** -0.5)
    H.assert_sparse(got, ref, mag, size, dtype, kind == U8, "large")
    assert (got[mag.sum(-1) == 0] == 0).all()
    assert wllm.device_errors() == 0


@pytest.mark.parametrize("dtype,kind,D,group", [(BF, BF, 128, 2), (F16, F16, 128, 12), (BF, BF, 256, 1), (F16, F16, 256, 3),
                                                (BF, U8, 256, 1), (F32, F32, 128, 1)])
def test_sparse_decode_of_more_lists_than_run_at_once(dtype, kind, D, group):
    """700 lists with a CTA each: 16-bit caches take the form with fewer stages, of which more fit an SM."""
    lens = [1 + 37 * i % 400 for i in range(175)]
    check_sparse(dtype, kind, D, 4 * group, 4, 16, lens, 9, D + group)


@pytest.mark.parametrize("dtype,kind,D,group", [(BF, BF, 128, 2), (F16, F16, 64, 4), (F16, F16, 256, 1), (F32, F32, 128, 4),
                                                (F32, F32, 64, 1), (F32, F32, 256, 1), (BF, U8, 128, 7), (F16, U8, 64, 9)])
def test_sparse_decode_of_lists_that_a_warp_looks_up_in_turns(dtype, kind, D, group):
    """80 blocks of 64 tokens are 320 units for the 2 or 4 warps of one CTA (32 at a lookup), in some 700 lists; a few rows
    are long and others end in the first lookup."""
    lens = [5120 - 3 * i if i % 8 == 0 else 64 * (i % 7) + 1 for i in range(175)]
    check_sparse(dtype, kind, D, 4 * group, 4, 64, lens, 80, 7 * D + group)


def test_sparse_decode_of_one_long_list_in_turns():
    """8 CTAs with 4 warps and more than 32 * 32 units."""
    check_sparse(BF, BF, 128, 8, 1, 256, [60000], 150, 3)
    check_sparse(F16, U8, 128, 8, 1, 256, [60000, 5], 150, 4)


@pytest.mark.parametrize("dtype,kind", [(BF, BF), (F16, U8), (F32, F32)])
@pytest.mark.parametrize("B", [2, 24, 32])
def test_selection_starts_long_rows_first(dtype, kind, B):
    """Up to 32 sequences of mixed, equal and zero lengths with more rows than CTAs run at once."""
    g = H.gen(B)
    Hkv, bs, D = 768 // B if B > 2 else 320, 16, 64
    choices = [0, 1, 500, 500, 3000, 3000, 3000, 1700, 64, 2999]
    lens = [choices[int(torch.randint(0, 10, (1,), generator=g))] for _ in range(B - 1)] + [3000]
    bt = shared_pool(g, lens, bs, 400)
    q = H.randn(g, B, Hkv, D, dtype=dtype)
    assert_selected(q, bounds_pool(g, 400, Hkv, D, kind), bt, i32(lens), Hkv, bs, 20, 1, 2)


@pytest.mark.parametrize("dtype,kind,D", [(BF, BF, 256), (F16, F16, 64), (BF, U8, 128), (F32, F32, 128)])
def test_selection_over_the_widest_table(dtype, kind, D):
    """30,720 blocks a sequence, the most that are taken: one row uses them all, others few; one block more is refused."""
    g = H.gen(D)
    bs, width, pool = 8, 30 * 1024, 900
    lens = [bs * width, 1234, bs * width - 5, 8 * 200]
    bt = shared_pool(g, lens, bs, pool)
    q = H.randn(g, 4, 4, D, dtype=dtype)
    kb = bounds_pool(g, pool, 2, D, kind)
    assert bt.shape[1] == width
    assert_selected(q, kb, bt, i32(lens), 2, bs, 64, 2, 3)
    wide = torch.zeros(4, width + 1, dtype=torch.int32)
    with pytest.raises(wllm.WllmError, match="at most"):
        assert_selected(q, kb, wide, i32(lens), 2, bs, 64, 2, 3)


def test_first_launches_race():
    """In a fresh process, threads make the first launches of one selection kernel at tables of several widths, some
    ascending and some descending, so that its shared-memory limit grows while others launch; each gives the bits that
    the same calls give one after another afterwards."""
    r = subprocess.run([sys.executable, "-c", """
import threading, torch
import paged_kv_cache_185_gb300 as wllm
g = torch.Generator().manual_seed(1)
widths = [600, 2000, 5000, 9000, 16000, 24000, 30 * 1024]
D, Hkv, pool, top = 64, 2, 500, 20
x = torch.randn(pool, Hkv, 2, D, generator=g)
kb = torch.stack([x.amin(2), x.amax(2)], 2).half().cuda()
calls = []
for w in widths:
    bt = torch.randint(0, pool, (2, w), generator=g, dtype=torch.int32).cuda()
    cl = torch.tensor([w * 8, w * 4 + 3], dtype=torch.int32).cuda()
    calls.append((torch.randn(2, 4, D, generator=g).half().cuda(), kb, bt, cl))
new = lambda: torch.full((2, Hkv, top), -7, dtype=torch.int32, device="cuda")
outs = [[new() for _ in widths] for _ in range(8)]
streams = [torch.cuda.Stream() for _ in outs]
gate, errors = threading.Barrier(len(outs)), []
torch.cuda.synchronize()
def work(i):
    try:
        order = list(range(len(widths)))
        order = order[::-1] if i % 2 else order[i // 2:] + order[:i // 2]
        with torch.cuda.stream(streams[i]):
            gate.wait()
            for k in order:
                wllm.select_blocks(outs[i][k], *calls[k], Hkv, 8, 1, 2)
            streams[i].synchronize()
    except Exception as e:
        errors.append(e)
threads = [threading.Thread(target=work, args=(i,)) for i in range(len(outs))]
[t.start() for t in threads]; [t.join() for t in threads]
assert not errors, errors
for k, c in enumerate(calls):
    want = wllm.select_blocks(new(), *c, Hkv, 8, 1, 2)
    torch.cuda.synchronize()
    assert (want >= 0).all()
    for o in outs:
        assert torch.equal(o[k], want), k
assert wllm.device_errors() == 0
"""], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


def last_blocks(g, pool, lens, bs, high):
    """Tables over the last blocks of a pool: (tables, the same tables into a small pool of those blocks, their ids)."""
    bt, n = H.block_tables(g, lens, bs, spare=0)
    ids = torch.arange(pool - n, pool, dtype=torch.int32) if high else torch.arange(n, dtype=torch.int32)
    return torch.where(bt < 0, bt, ids[bt.clamp(min=0).long()]), bt, ids.long()


def test_a_step_at_offsets_beyond_32_bits():
    """Caches of 2.3e9 elements each: the rotary append, the bounds, the choice and the attention on their last blocks."""
    g = H.gen(77)
    Hq, Hkv, D, bs, top = 16, 8, 128, 16, 6
    pool = 140_000
    assert pool * Hkv * bs * D > 2 ** 31
    lens = [200, 31, 333]
    bt, small, ids = last_blocks(g, pool, lens, bs, True)
    kc, vc = (torch.empty(pool, Hkv, bs, D, dtype=BF, device="cuda") for _ in range(2))
    kb = torch.zeros(pool, Hkv, 2, D, dtype=BF, device="cuda")
    T = sum(lens)
    pos = torch.cat([torch.arange(n) for n in lens])
    seq = torch.arange(3).repeat_interleave(torch.tensor(lens))
    slots = bt[seq, pos // bs].long() * bs + pos % bs
    assert slots.min() > (pool - len(ids) - 1) * bs
    q, k, v = (H.randn(g, T, n, D, dtype=BF) for n in (Hq, Hkv, Hkv))
    table = H.rotary_table(400, D)
    out_q = torch.empty(T, Hq, D, dtype=BF, device="cuda")
    wllm.rotate_and_cache(out_q, q.cuda(), k.cuda(), v.cuda(), kc, vc, slots.cuda(), pos.cuda(), table.cuda())
    btd, cl = bt.cuda(), i32(lens).cuda()
    qsl = i32([0] + lens).cumsum(0).to(torch.int32)
    wllm.update_key_bounds(kb, kc, btd, cl, bs, query_start_loc=qsl.cuda())
    last = out_q[(qsl[1:] - 1).long().cuda()].contiguous()
    sel = torch.empty(3, Hkv, top, dtype=torch.int32, device="cuda")
    wllm.select_blocks(sel, last, kb, btd, cl, Hkv, bs, 1, 2)
    out = wllm.paged_attention_decode_sparse(torch.empty_like(last), last, kc, vc, btd, cl, sel, Hkv, 0.1, bs)
    torch.cuda.synchronize()
    assert wllm.device_errors() == 0
    skc, svc, skb = (x[ids.cuda()].cpu() for x in (kc, vc, kb))
    rows = skc[(slots // bs - ids[0]), :, slots % bs]
    H.assert_turned(rows, *S.rotate_rows(k, pos, table), BF, "keys")
    assert torch.equal(H.bits(svc[(slots // bs - ids[0]), :, slots % bs]), H.bits(v))
    full = S.key_bounds(skc, small, i32(lens), lens, S.values(torch.zeros_like(skb)))
    assert torch.equal(S.values(skb), full)
    want = S.select_blocks(last.cpu(), skb, small, i32(lens), Hkv, bs, top, 1, 2)
    assert torch.equal(sel.cpu(), want)
    H.assert_sparse(out.cpu(), *S.sparse_decode(last.cpu(), skc, svc, small, i32(lens), want, float(torch.tensor(0.1))), BF, False, "end")


def test_bounds_and_choice_at_byte_offsets_beyond_32_bits():
    """9 million blocks of E4M3 codes: 4.6 GB of bounds, 18 GB of keys."""
    g = H.gen(78)
    D, bs, pool, top = 256, 8, 9_000_000, 9
    assert pool * 2 * D > 2 ** 32
    lens = [8 * 100, 8 * 40 + 3]
    bt, small, ids = last_blocks(g, pool, lens, bs, True)
    kc = torch.empty(pool, 1, bs, D, dtype=U8, device="cuda")
    kb = torch.empty(pool, 1, 2, D, dtype=U8, device="cuda")
    host = H.cache(g, len(ids), 1, bs, D, U8)
    kc[ids.cuda()] = host.cuda()
    kb[ids.cuda()] = 0
    btd, cl = bt.cuda(), i32(lens).cuda()
    wllm.update_key_bounds(kb, kc, btd, cl, bs, query_start_loc=i32([0, lens[0], sum(lens)]).cuda())
    q = H.randn(g, 2, 4, D, dtype=F16)
    sel = torch.empty(2, 1, top, dtype=torch.int32, device="cuda")
    wllm.select_blocks(sel, q.cuda(), kb, btd, cl, 1, bs, 1, 2)
    torch.cuda.synchronize()
    skb = kb[ids.cuda()].cpu()
    assert torch.equal(S.values(skb), S.key_bounds(host, small, i32(lens), lens, S.values(torch.zeros_like(skb))))
    assert torch.equal(sel.cpu(), S.select_blocks(q, skb, small, i32(lens), 1, bs, top, 1, 2))
    assert wllm.device_errors() == 0
