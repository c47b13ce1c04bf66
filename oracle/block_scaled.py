"""Definitions of slot assignment, the block-scaled append and the attention over a block-scaled cache.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Host tensors in, host tensors out; plain loops, torch float64
operations and (where a definition is in binary32) float32 ones, sharing no code with the CUDA path.
"""
from __future__ import annotations

import math

import torch

from . import e4m3_encode, widen, widen_e4m3

__all__ = ["assign_slots", "block_scale", "append", "attention"]

LEAST, MOST = 2.0 ** -40, 2.0 ** 40


def assign_slots(block_tables, context_lens, new_tokens, free_blocks, num_free, rows, block_size):
    """(slots, positions, starts, lengths, count, tables, stack) after the call, of valid arguments but for negative
    entries in rows that are given back."""
    table, lens, stack = block_tables.clone(), context_lens.tolist(), free_blocks.tolist()
    new, count, width = new_tokens.tolist(), int(num_free), block_tables.shape[1]
    blocks = lambda n: -(-n // block_size)  # noqa: E731
    for b, n in enumerate(new):
        if n < 0:
            for k in range(blocks(lens[b])):
                if int(table[b, k]) >= 0:
                    stack[count] = int(table[b, k])
                    count += 1
            lens[b] = 0
    slots, positions, starts = [], [], [0]
    asked_tokens = asked_blocks = used = 0
    for b, n in enumerate(new):
        got = 0
        if n >= 0 and lens[b] + n <= width * block_size:
            held, need = blocks(lens[b]), blocks(lens[b] + n) - blocks(lens[b])
            asked_tokens += n
            asked_blocks += need
            if asked_tokens <= rows and (need == 0 or asked_blocks <= count):
                got = n
                for k in range(need):
                    table[b, held + k] = stack[count - 1 - used]
                    used += 1
                for p in range(lens[b], lens[b] + n):
                    slots.append(int(table[b, p // block_size]) * block_size + p % block_size)
                    positions.append(p)
                lens[b] += n
        starts.append(starts[-1] + got)
    pad = rows - len(slots)
    return (torch.tensor(slots + [-1] * pad, dtype=torch.int64), torch.tensor(positions + [0] * pad, dtype=torch.int64),
            torch.tensor(starts, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32), count - used, table,
            torch.tensor(stack, dtype=torch.int32))


def block_scale(x):
    """The scale that new elements x need: 2^e, the least e in [-40, 40] with every finite |x| <= 448 2^e."""
    y = widen(x).abs()
    m = y[torch.isfinite(y)].max().item() if torch.isfinite(y).any() else 0.0
    e = -40
    while e < 40 and m > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(key, value, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, query_start_loc=None):
    """Writes codes and scales of the new tokens into host caches (uint8 [N_b,Hkv,bs,D]) and scales, in place."""
    bs = k_cache.shape[2]
    for b, L in enumerate(context_lens.tolist()):
        if query_start_loc is None:
            row, n = b, min(L, 1)
        else:
            row, n = int(query_start_loc[b]), int(query_start_loc[b + 1] - query_start_loc[b])
        p = L - n
        while p < L:
            j, off = p // bs, p % bs
            count = min(bs - off, L - p)
            i = int(block_tables[b, j])
            for x, cache, scales in ((key, k_cache, k_scales), (value, v_cache, v_scales)):
                for h in range(x.shape[1]):
                    new = x[row:row + count, h]
                    scale = torch.tensor(block_scale(new), dtype=torch.float32)
                    if off:
                        old = scales[i, h].clone()
                        old = torch.tensor(LEAST, dtype=torch.float32) if old.isnan() else old.clamp(LEAST, MOST)
                        scale = torch.maximum(scale, old)
                        if scale > old:
                            f = old * (1.0 / scale)
                            cache[i, h, :off] = e4m3_encode(widen_e4m3(cache[i, h, :off]).float() * f)
                    scales[i, h] = scale
                    cache[i, h, off:off + count] = e4m3_encode(new.float() * (1.0 / scale))
            p, row = p + count, row + count


def attention(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale, query_start_loc=None):
    """(float64 out [T,Hq,D]; float64 [T,Hq,D] sum_t p_t |v_t|; float64 [T,Hq] largest |scale| sum_d |q_d k_td|; float64
    [T,Hq] tokens times the largest value scale): the attention, and the sizes that scale its rounding errors."""
    qd, ks, vs = widen(q), k_scales.double().clamp(LEAST, MOST), v_scales.double().clamp(LEAST, MOST)
    T, Hq, D = qd.shape
    Hkv, bs = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    out, mag = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    size, least = torch.zeros(T, Hq, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    for b, L in enumerate(context_lens.tolist()):
        r0, r1 = (b, b + 1) if query_start_loc is None else (int(query_start_loc[b]), int(query_start_loc[b + 1]))
        if L == 0 or r0 == r1:
            continue
        n = -(-L // bs)
        ids = block_tables[b, :n].long()
        pos = torch.arange(L - (r1 - r0), L) if query_start_loc is not None else torch.tensor([L - 1])
        for h in range(Hkv):
            k = (widen_e4m3(k_cache[ids, h]) * ks[ids, h][:, None, None]).reshape(-1, D)[:L]
            v = (widen_e4m3(v_cache[ids, h]) * vs[ids, h][:, None, None]).reshape(-1, D)[:L]
            hidden = torch.arange(L)[None, :] > pos[:, None]
            for g in range(h * G, (h + 1) * G):
                s = (qd[r0:r1, g] @ k.T) * scale
                p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
                out[r0:r1, g], mag[r0:r1, g] = p @ v, p @ v.abs()
                size[r0:r1, g] = ((qd[r0:r1, g].abs() @ k.abs().T).masked_fill(hidden, 0.0)).max(-1).values * abs(scale)
                least[r0:r1, g] = (pos + 1).double() * vs[ids, h].max()
    return out, mag, size, least
