"""Definitions of the rotary append, key bounds, block selection and block-sparse decode in binary64.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Host tensors in, float64 out; plain loops and torch
float64 operations, sharing no code with the CUDA path.
"""
from __future__ import annotations

import torch

from . import widen, widen_e4m3

__all__ = ["values", "rotate_rows", "key_bounds", "scores", "select_blocks", "sparse_decode"]


def values(x: torch.Tensor) -> torch.Tensor:
    """Stored elements (f32, f16, bf16, or E4M3 codes as uint8) as float64."""
    return widen_e4m3(x) if x.dtype == torch.uint8 else widen(x)


def rotate_rows(x, positions, cos_sin, weight=None, eps=1e-6, style="halves", sections=None):
    """x [T,H,D] -> (float64 [T,H,D] normalised and turned, float64 of the same shape: the length of each element's
    pair, which scales the rounding errors of a turn)."""
    y = values(x)
    T, H, D = y.shape
    if weight is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + float(torch.tensor(eps, dtype=torch.float32))) * values(weight)
    table = cos_sin.double()
    pairs = table.shape[1] // 2
    pos = positions.view(len(sections) if sections else 1, T)
    axis_of = [a for a, n in enumerate(sections if sections else [pairs]) for _ in range(n)]
    out, size = y.clone(), y.abs()
    for p in range(pairs):
        i, j = (p, p + pairs) if style == "halves" else (2 * p, 2 * p + 1)
        row = table[pos[axis_of[p]]]
        c, s = row[:, p:p + 1], row[:, pairs + p:pairs + p + 1]
        a, b = y[..., i], y[..., j]
        out[..., i], out[..., j] = a * c - b * s, b * c + a * s
        size[..., i] = size[..., j] = torch.sqrt(a * a + b * b)
    return out, size


def key_bounds(k_cache, block_tables, context_lens, new, old):
    """``old`` (float64 [N_b,Hkv,2,D]) with the bounds of every block that the last new[b] tokens filled."""
    k, out, bs = values(k_cache), old.clone(), k_cache.shape[2]
    for b, n in enumerate(context_lens.tolist()):
        for j in range((n - int(new[b])) // bs, n // bs):
            i = int(block_tables[b, j])
            out[i, :, 0], out[i, :, 1] = k[i].amin(1), k[i].amax(1)
    return out


def scores(q, bounds, block_tables, context_lens, num_kv_heads, block_size):
    """Per sequence a float64 [Hkv, n]: sum over the group's heads and dims of max(q lo, q hi); a NaN, as with a NaN or
    infinite bound, counts as +inf."""
    qd, bd = values(q), values(bounds)
    G = q.shape[1] // num_kv_heads
    got = []
    for b, L in enumerate(context_lens.tolist()):
        n = -(-L // block_size)
        x = bd[block_tables[b, :n].long()]                        # [n, Hkv, 2, D]
        lo, hi = x[:, :, 0], x[:, :, 1]
        s = torch.zeros(num_kv_heads, n, dtype=torch.float64)
        for h in range(num_kv_heads):
            for g in range(G):
                v = qd[b, h * G + g]
                # max(q lo, q hi) for lo <= hi; zero times an infinite bound is NaN
                s[h] += (v.clamp(min=0) * hi[:, h] + v.clamp(max=0) * lo[:, h]).sum(-1)
        got.append(torch.where(s.isnan(), torch.full_like(s, float("inf")), s))
    return got


def select_blocks(q, bounds, block_tables, context_lens, num_kv_heads, block_size, top, num_sink, num_recent):
    out = torch.full((q.shape[0], num_kv_heads, top), -1, dtype=torch.int32)
    for b, s in enumerate(scores(q, bounds, block_tables, context_lens, num_kv_heads, block_size)):
        n = s.shape[1]
        for h in range(num_kv_heads):
            if n <= top:
                ids = list(range(n))
            else:
                fixed = list(range(num_sink)) + list(range(n - num_recent, n))
                row = s[h].tolist()
                rest = sorted(range(num_sink, n - num_recent), key=lambda j: (-row[j], j))[:top - len(fixed)]
                ids = sorted(fixed + rest)
            out[b, h, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
    return out


def sparse_decode(q, k_cache, v_cache, block_tables, context_lens, selected, scale, k_scale=1.0, v_scale=1.0):
    """(float64 out [B,Hq,D]; float64 [B,Hq,D] sum_t p_t |v_t|; float64 [B,Hq] largest scale * sum_d |q_d k_td|): the
    attention over the listed blocks, and the sizes that scale its rounding errors."""
    qd, k, v = values(q), values(k_cache) * k_scale, values(v_cache) * v_scale
    B, Hq, D = qd.shape
    Hkv, bs = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out, mag = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    size = torch.zeros(B, Hq, dtype=torch.float64)
    for b, L in enumerate(context_lens.tolist()):
        for h in range(Hkv):
            at = [j * bs + i for j in selected[b, h].tolist() if j >= 0 for i in range(bs) if j * bs + i < L]
            if not at:
                continue
            t = torch.tensor(at)
            blk = block_tables[b].long()[t // bs]
            kk, vv = k[blk, h, t % bs], v[blk, h, t % bs]
            for g in range(h * G, (h + 1) * G):
                p = torch.softmax(kk @ qd[b, g] * scale, 0)
                out[b, g], mag[b, g] = p @ vv, p @ vv.abs()
                size[b, g] = (kk.abs() @ qd[b, g].abs()).max() * abs(scale)
    return out, mag, size
