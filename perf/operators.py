"""Cases that measure the rotary append and the block-sparse decode of the library.

Four operators make one layer's decode step over a paged cache of which only the blocks that matter are read:

  rotate   rotate_and_cache: per-head norms of query and key, rotary positions (one or several axes), query written
           out, key and value written to their cache slots
  bounds   update_key_bounds: elementwise minimum and maximum of the keys of every block that new tokens filled
  select   select_blocks: the blocks whose bounds allow the largest scores, for each sequence and kv head
  sparse   paged_attention_decode_sparse: attention over the selected blocks

``run`` with ``own`` false is the plain form in elementary torch operations; with ``own`` true it is the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}
DEVICE = "cuda"
EPS = 1e-6
K_SCALE, V_SCALE = 0.03125, 0.025  # an fp8 cache's scales: codes of values up to a few units use the format's range


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a few interactive requests: the call's own latency
        dict(name="rotate step of 4", op="rotate", seqs=4, tokens=4, q_heads=32, kv_heads=8, dim=128, rot=128, block=16,
             dtype="bf16", cache="bf16", norm=True, axes=1, style="halves", padded=0),
        # one decode step of a full batch, padded to its captured size
        dict(name="rotate step of 256", op="rotate", seqs=251, tokens=251, q_heads=28, kv_heads=4, dim=128, rot=128,
             block=16, dtype="bf16", cache="bf16", norm=True, axes=1, style="halves", padded=5),
        # prompts with images: three position axes
        dict(name="rotate prompts axes", op="rotate", seqs=5, tokens=8192, q_heads=28, kv_heads=4, dim=128, rot=128,
             block=16, dtype="bf16", cache="bf16", norm=True, axes=3, style="halves", padded=0),
        # an odd chunk into an fp8 cache, half of the head rotated, neighbours paired, no norms
        dict(name="rotate chunk fp8", op="rotate", seqs=3, tokens=3001, q_heads=32, kv_heads=8, dim=128, rot=64, block=16,
             dtype="f16", cache="fp8", norm=False, axes=1, style="adjacent", padded=0),
        # the bounds of freshly cached prompts
        dict(name="bounds prompts", op="bounds", seqs=16, lo=1500, hi=6000, chunk=2048, kv_heads=8, dim=128, block=16,
             cache="bf16"),
        # one decode step: a sixteenth of the sequences fill a block
        dict(name="bounds step of 256", op="bounds", seqs=256, lo=128, hi=4000, chunk=1, kv_heads=4, dim=128, block=16,
             cache="bf16"),
        # a single long chat
        dict(name="select one 16K", op="select", seqs=1, lo=16000, hi=16000, q_heads=32, kv_heads=4, dim=64, block=16,
             dtype="f16", cache="f16", top=64, sink=1, recent=2),
        # long documents
        dict(name="select 8 long", op="select", seqs=8, lo=32768, hi=131072, q_heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16", cache="bf16", top=128, sink=1, recent=4),
        # a busy server over an fp8 cache
        dict(name="select 64 fp8", op="select", seqs=64, lo=3000, hi=24000, q_heads=28, kv_heads=4, dim=128, block=16,
             dtype="bf16", cache="fp8", top=96, sink=4, recent=8),
        # a single long chat
        dict(name="sparse one 16K", op="sparse", seqs=1, lo=16000, hi=16000, q_heads=32, kv_heads=4, dim=64, block=16,
             dtype="f16", cache="f16", top=64),
        # long documents
        dict(name="sparse 8 long", op="sparse", seqs=8, lo=32768, hi=131072, q_heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16", cache="bf16", top=128),
        # a busy server over an fp8 cache
        dict(name="sparse 256 fp8", op="sparse", seqs=256, lo=1000, hi=8000, q_heads=28, kv_heads=4, dim=128, block=16,
             dtype="bf16", cache="fp8", top=96),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rotate", "bounds", "select", "sparse"])
    group, kv_heads = rng.choice([(1, 8), (1, 32), (4, 8), (7, 4), (8, 4), (8, 1), (16, 2), (5, 2), (3, 5)])
    dim, block = rng.choice([64, 128, 128, 256]), rng.choice([8, 16, 16, 32, 64])
    dtype = rng.choice(["bf16", "f16", "bf16", "f32"])
    cache = "fp8" if dtype != "f32" and rng.random() < 0.35 else dtype
    if cache == "fp8" and dim == 64:
        block = max(block, 16)
    row = kv_heads * dim * BYTES[cache]  # bytes of one token's keys
    case = dict(op=op, seqs=0, q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim, block=block, dtype=dtype, cache=cache)
    if op == "rotate":
        most = max(64, int(1.3e8 / ((2 * group + 4) * kv_heads * dim * BYTES[dtype])))
        tokens = spread(rng, 1, min(most, 8192))
        seqs = tokens if tokens <= 512 and rng.random() < 0.6 else spread(rng, 1, min(tokens, 40))
        axes = rng.choice([1, 1, 2, 3])
        case.update(seqs=seqs, tokens=tokens, rot=rng.choice([dim, dim, dim // 2]), norm=rng.random() < 0.7, axes=axes,
                    style=rng.choice(["halves", "halves", "adjacent"]), padded=rng.choice([0, 0, 3]))
        return case
    if op == "bounds":
        del case["q_heads"], case["dtype"]
        chunk = rng.choice([1, spread(rng, 2, 4096)])
        seqs = spread(rng, 1, 300)
        seqs = max(1, min(seqs, int(6.5e7 / (chunk * row)))) if chunk > 1 else seqs
        lo = spread(rng, 1, 4000)
        hi = max(lo, min(spread(rng, lo, 20000), int(2.5e8 / (seqs * row))))
        case.update(seqs=seqs, lo=lo, hi=hi, chunk=chunk)
        return case
    top = spread(rng, 8, 160)
    if op == "select":
        need = 3 * top * block  # the longest sequence has blocks to leave out
        seqs = max(1, min(spread(rng, 1, 128), int(1.4e8 * block / (2 * row * need))))
        hi = spread(rng, need, max(need, min(131072, int(1.4e8 * block / (2 * row * seqs)))))
        lo = hi if seqs == 1 else spread(rng, 1, hi)
        sink = rng.choice([0, 1, 4])
        case.update(seqs=seqs, lo=lo, hi=hi, top=top, sink=sink, recent=rng.randint(1, max(1, top - sink - 1) // 2 + 1))
        return case
    seqs = max(1, min(spread(rng, 1, 256), int(3.5e8 / (2 * row * top * block)),
                      int(5e9 / (4 * case["q_heads"] * dim * top * block))))
    lo = spread(rng, 1, 30000)
    lo = max(1, min(lo, int(1e9 / (row * seqs))))
    hi = max(lo, min(spread(rng, lo, 131072), int(1e9 / (row * seqs))))
    case.update(seqs=seqs, lo=lo, hi=hi, top=top)
    return case


# ---------------------------------------------------------------- sizes that follow from a case alone
def ragged(count, lo, hi):
    """`count` lengths spread evenly over lo..hi, in an order without pattern."""
    return [lo + int((hi - lo + 1) * ((0.5 + 0.6180339887498949 * i) % 1.0)) for i in range(count)]


def chunks(case):
    """Tokens of each sequence of a rotate case: they sum to case["tokens"]."""
    n, t = case["seqs"], case["tokens"]
    if t == n:
        return [1] * n
    w = [1 + (0.5 + 0.6180339887498949 * i) % 1.0 for i in range(n)]
    ends = [round(t * sum(w[:i + 1]) / sum(w)) for i in range(n)]
    return [b - a for a, b in zip([0] + ends, ends)]


def sections(case):
    pairs, axes = case["rot"] // 2, case["axes"]
    return {1: [pairs], 2: [pairs // 4, pairs - pairs // 4],
            3: [pairs // 4, 3 * pairs // 8, pairs - pairs // 4 - 3 * pairs // 8]}[axes]


def work(case):
    d, bs, hkv, c = case["dim"], case["block"], case["kv_heads"], BYTES[case["cache"]]
    if case["op"] == "rotate":
        t, e, hq = case["tokens"], BYTES[case["dtype"]], case["q_heads"]
        values = t * (hq + 2 * hkv) * d
        return {"bytes": values * e + t * hq * d * e + 2 * t * hkv * d * c + t * (8 + 8 * case["axes"] + 4 * case["rot"]),
                "flops": values * (3 * case["norm"] + 3)}
    lens = ragged(case["seqs"], case["lo"], case["hi"])
    if case["op"] == "bounds":
        full = sum(n // bs - (n - min(n, case["chunk"])) // bs for n in lens)
        return {"bytes": full * (hkv * (bs + 2) * d * c + 4) + 8 * len(lens), "flops": full * hkv * bs * d * 2}
    e, hq, top = BYTES[case["dtype"]], case["q_heads"], case["top"]
    blocks = [-(-n // bs) for n in lens]
    if case["op"] == "select":
        scored = sum(n - case["sink"] - case["recent"] for n in blocks if n > top)
        return {"bytes": scored * (hkv * 2 * d * c + 4) + len(lens) * (hq * d * e + hkv * top * 4 + 4), "flops": scored * hkv * 2 * d * 2}
    tokens = sum(min(n, min(b, top) * bs) for n, b in zip(lens, blocks))
    return {"bytes": tokens * hkv * 2 * d * c + 2 * len(lens) * hq * d * e + sum(min(b, top) for b in blocks) * (hkv + 1) * 4,
            "flops": tokens * hq * d * 4}


# ---------------------------------------------------------------- inputs
def normal(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEVICE) * scale).to(dtype)


def tables(gen, counts, width=None):
    """Block tables for sequences of `counts` blocks out of a shuffled pool (-1 past a sequence's last), and the pool's size."""
    width = max(counts) if width is None else width
    used = sum(counts)
    pool = used + 3
    order = torch.randperm(pool, generator=gen, device=DEVICE)[:used].to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEVICE)
    at = torch.arange(width, device=DEVICE)[None, :]
    table[at < torch.tensor(counts, device=DEVICE)[:, None]] = order
    return table, pool


def keys(gen, shape, cache, scale):
    """Cached keys as they come: a bias for each channel, a drift from block to block, and noise; [blocks, heads, tokens, dim]."""
    n, h, bs, d = shape
    bias = torch.randn(h, 1, d, generator=gen, device=DEVICE)
    drift = torch.randn(n, h, 1, d, generator=gen, device=DEVICE) * 0.5
    k = torch.empty(shape, dtype=DTYPES[cache], device=DEVICE)
    for a in range(0, n, 4096):
        x = torch.randn(min(4096, n - a), h, bs, d, generator=gen, device=DEVICE) + drift[a:a + 4096] + bias
        k[a:a + 4096] = (x / scale).to(k.dtype)
    return k


def values(gen, shape, cache, scale):
    v = torch.empty(shape, dtype=DTYPES[cache], device=DEVICE)
    for a in range(0, shape[0], 4096):
        v[a:a + 4096] = (torch.randn(min(4096, shape[0] - a), *shape[1:], generator=gen, device=DEVICE) / scale).to(v.dtype)
    return v


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    d, bs, hkv, c = case["dim"], case["block"], case["kv_heads"], case["cache"]
    fp8 = c == "fp8"
    s = {"case": case, "fp8": fp8, "block_size": bs, "k_scale": K_SCALE if fp8 else 1.0, "v_scale": V_SCALE if fp8 else 1.0}
    if case["op"] == "rotate":
        return prepare_rotate(s, case, gen)
    lens = ragged(case["seqs"], case["lo"], case["hi"])
    lens = [lens[i] for i in torch.randperm(len(lens), generator=gen, device=DEVICE).tolist()]
    blocks = [-(-n // bs) for n in lens]
    s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    s["block_tables"], pool = tables(gen, blocks)
    if case["op"] == "bounds":
        s["k_cache"] = keys(gen, (pool, hkv, bs, d), c, s["k_scale"])
        s["key_bounds"] = normal(gen, pool, hkv, 2, d, dtype=DTYPES[c])  # what these blocks held before
        new = torch.tensor([0] + [min(n, case["chunk"]) for n in lens], device=DEVICE)
        s["query_start_loc"] = None if case["chunk"] == 1 else new.cumsum(0).to(torch.int32)
        s["new"] = new[1:]
        return s
    dt = DTYPES[case["dtype"]]
    s["q"] = normal(gen, len(lens), case["q_heads"], d, dtype=dt)
    if case["op"] == "select":
        s["key_bounds"] = torch.empty(pool, hkv, 2, d, dtype=DTYPES[c], device=DEVICE)
        for a in range(0, pool, 4096):
            k = keys(gen, (min(4096, pool - a), hkv, bs, d), c, s["k_scale"]).float()
            s["key_bounds"][a:a + 4096] = torch.stack([k.amin(2), k.amax(2)], 2).to(DTYPES[c])
        s["selected"] = torch.empty(len(lens), hkv, case["top"], dtype=torch.int32, device=DEVICE)
        return s
    s["k_cache"] = keys(gen, (pool, hkv, bs, d), c, s["k_scale"])
    s["v_cache"] = values(gen, (pool, hkv, bs, d), c, s["v_scale"])
    s["out"] = torch.empty_like(s["q"])
    s["scale"] = 1.0 / math.sqrt(d)
    # a selection as the select operator leaves it: ascending, the last block in it, -1 behind a short one
    top, most = case["top"], max(blocks)
    n = torch.tensor(blocks, device=DEVICE)[:, None, None]
    rank = torch.rand(len(lens), hkv, most, generator=gen, device=DEVICE)
    at = torch.arange(most, device=DEVICE)
    rank = torch.where(at == n - 1, 2.0, torch.where(at < n, rank, -1.0))
    kept = rank.topk(min(top, most), dim=2)
    ids = torch.where(kept.values < 0, most, kept.indices).sort(dim=2).values
    s["selected"] = torch.full((len(lens), hkv, top), -1, dtype=torch.int32, device=DEVICE)
    s["selected"][:, :, :ids.shape[2]] = torch.where(ids == most, -1, ids)
    return s


def prepare_rotate(s, case, gen):
    d, bs, hkv, hq, rot, t = case["dim"], case["block"], case["kv_heads"], case["q_heads"], case["rot"], case["tokens"]
    dt, count = DTYPES[case["dtype"]], chunks(case)
    far = 32768
    first = torch.randint(0, far - 8192, (len(count),), generator=gen, device=DEVICE)
    table, pool = tables(gen, [-(-(bs - 1 + n) // bs) for n in count])  # room for any first position
    n = torch.tensor(count, device=DEVICE)
    seq = torch.arange(len(count), device=DEVICE).repeat_interleave(n, output_size=t)
    within = torch.arange(t, device=DEVICE) - (n.cumsum(0) - n)[seq]
    place = (first % bs)[seq] + within
    slots = table[seq, place // bs].long() * bs + place % bs
    pos = first[seq] + within
    pad = case["padded"]
    s["slot_mapping"] = torch.cat([slots, slots.new_full((pad,), -1)])
    pos = torch.cat([pos, pos.new_zeros(pad)])
    if case["axes"] > 1:  # time, then height (and width) of an image's tiles
        grid = torch.randint(0, 256, (case["axes"] - 1, t + pad), generator=gen, device=DEVICE)
        pos = torch.cat([pos[None], grid])
    s["positions"] = pos
    fused = normal(gen, t + pad, (hq + 2 * hkv) * d, dtype=dt)  # a fused projection's output, in slices
    s["q"] = fused[:, :hq * d].view(t + pad, hq, d)
    s["key"] = fused[:, hq * d:(hq + hkv) * d].view(t + pad, hkv, d)
    s["value"] = fused[:, (hq + hkv) * d:].view(t + pad, hkv, d)
    s["q_out"] = normal(gen, t + pad, hq, d, dtype=dt)
    s["k_cache"] = values(gen, (pool, hkv, bs, d), case["cache"], s["k_scale"])
    s["v_cache"] = values(gen, (pool, hkv, bs, d), case["cache"], s["v_scale"])
    freq = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
    angle = torch.arange(far, dtype=torch.float64, device=DEVICE)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["q_weight"] = (1 + normal(gen, d, scale=0.2)).to(dt) if case["norm"] else None
    s["k_weight"] = (1 + normal(gen, d, scale=0.2)).to(dt) if case["norm"] else None
    s["sections"] = sections(case) if case["axes"] > 1 else None
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return (run_own if own else run_plain)(s)


def run_own(s):
    import paged_kv_cache_185_gb300 as wllm
    case = s["case"]
    if case["op"] == "rotate":
        args = [s[k] for k in ("q_out", "q", "key", "value", "k_cache", "v_cache", "slot_mapping", "positions", "cos_sin")]
        how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, style=case["style"], sections=s["sections"])
        if s["fp8"]:
            wllm.rotate_and_cache_fp8(*args, s["k_scale"], s["v_scale"], **how)
        else:
            wllm.rotate_and_cache(*args, **how)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if case["op"] == "bounds":
        wllm.update_key_bounds(s["key_bounds"], s["k_cache"], s["block_tables"], s["context_lens"], s["block_size"],
                               query_start_loc=s["query_start_loc"])
        return {"key_bounds": s["key_bounds"]}
    if case["op"] == "select":
        wllm.select_blocks(s["selected"], s["q"], s["key_bounds"], s["block_tables"], s["context_lens"], case["kv_heads"],
                           s["block_size"], num_sink=case["sink"], num_recent=case["recent"])
        return {"selected": s["selected"]}
    args = [s[k] for k in ("out", "q", "k_cache", "v_cache", "block_tables", "context_lens", "selected")]
    if s["fp8"]:
        wllm.paged_attention_decode_sparse_fp8(*args, case["kv_heads"], s["scale"], s["k_scale"], s["v_scale"], s["block_size"])
    else:
        wllm.paged_attention_decode_sparse(*args, case["kv_heads"], s["scale"], s["block_size"])
    return {"out": s["out"]}


def run_plain(s):
    return {"rotate": plain_rotate, "bounds": plain_bounds, "select": plain_select, "sparse": plain_sparse}[s["case"]["op"]](s)


def bits(x):
    """The same storage as whole numbers, for indexed writes of any element type."""
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


def stored(x, like, scale, fp8):
    """32-bit values as the cache holds them."""
    return (x * (1.0 / scale)).clamp(-448.0, 448.0).to(like.dtype) if fp8 else x.to(like.dtype)


def plain_rotate(s):
    case = s["case"]
    rot, pairs = case["rot"], case["rot"] // 2
    if case["axes"] > 1:
        axis = torch.arange(case["axes"], device=DEVICE).repeat_interleave(torch.tensor(s["sections"], device=DEVICE))
        pos = s["positions"][axis].T  # [T, pairs]
    else:
        pos = s["positions"][:, None].expand(-1, pairs)
    at = torch.arange(pairs, device=DEVICE)
    cos, sin = s["cos_sin"][pos, at][:, None, :], s["cos_sin"][pos, pairs + at][:, None, :]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        if case["style"] == "halves":
            a, b = x[..., :pairs], x[..., pairs:rot]
            return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)

    slots, bs = s["slot_mapping"], s["block_size"]
    live = slots >= 0
    s["q_out"].copy_(torch.where(live[:, None, None], turned(s["q"], s["q_weight"]).to(s["q_out"].dtype), s["q_out"]))
    blk, off = slots[live] // bs, slots[live] % bs
    for name, rows in (("k", turned(s["key"], s["k_weight"])), ("v", s["value"].float())):
        cache = s[name + "_cache"]
        bits(cache)[blk, :, off] = bits(stored(rows[live], cache, s[name + "_scale"], s["fp8"]))
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def plain_bounds(s):
    lens, bs = s["context_lens"].long(), s["block_size"]
    at = torch.arange(s["block_tables"].shape[1], device=DEVICE)[None, :]
    filled = (at >= ((lens - s["new"]) // bs)[:, None]) & (at < (lens // bs)[:, None])
    ids = s["block_tables"][filled].long()
    k = bits(s["k_cache"])[ids].view(s["k_cache"].dtype).float()
    bits(s["key_bounds"])[ids] = bits(torch.stack([k.amin(2), k.amax(2)], 2).to(s["key_bounds"].dtype))
    return {"key_bounds": s["key_bounds"]}


def plain_select(s):
    case, q, lens = s["case"], s["q"], s["context_lens"].long()
    (b, hq, d), hkv, bs, top = q.shape, case["kv_heads"], s["block_size"], case["top"]
    n = ((lens + bs - 1) // bs)[:, None, None]
    width = s["block_tables"].shape[1]
    # in 64 bits: two blocks' scores can lie next to one another at the border
    heads = q.double().view(b, hkv, hq // hkv, d)
    up, down = heads.clamp(min=0).sum(2), heads.clamp(max=0).sum(2)
    ids = s["block_tables"].long().clamp(min=0)
    both = bits(s["key_bounds"])[ids].view(s["key_bounds"].dtype)  # [B, width, Hkv, 2, D]
    score = torch.einsum("bhd,bjhd->bhj", up, both[:, :, :, 1].double())
    score += torch.einsum("bhd,bjhd->bhj", down, both[:, :, :, 0].double())
    at = torch.arange(width, device=DEVICE)
    inf = float("inf")
    score = torch.where(score.isnan(), inf, score)
    # the first and the last blocks come before any score, and what is behind the sequence after all
    first = torch.where((at < case["sink"]) | (at >= n - case["recent"]), 0, 1).expand_as(score)
    first = torch.where(at < n, first, 2)
    order = score.sort(dim=2, descending=True, stable=True).indices
    order = order.gather(2, first.gather(2, order).sort(dim=2, stable=True).indices)[:, :, :top]
    ids = torch.where(order < n, order, width).sort(dim=2).values
    s["selected"].fill_(-1)
    s["selected"][:, :, :ids.shape[2]] = torch.where(ids == width, -1, ids).to(torch.int32)
    return {"selected": s["selected"]}


def plain_sparse(s):
    case, q, chosen = s["case"], s["q"], s["selected"].long()
    (b, hq, d), hkv, bs = q.shape, case["kv_heads"], s["block_size"]
    ids = s["block_tables"].long().gather(1, chosen.clamp(min=0).view(b, -1)).view(b, hkv, -1)
    at = chosen[..., None] * bs + torch.arange(bs, device=DEVICE)
    live = ((chosen[..., None] >= 0) & (at < s["context_lens"][:, None, None, None])).view(b, hkv, 1, -1)
    head = torch.arange(hkv, device=DEVICE)[None, :, None]

    def rows(cache, scale):
        x = bits(cache)[ids, head].view(cache.dtype).view(b, hkv, -1, d).float()
        return torch.where(live.transpose(2, 3), x * scale, 0.0)

    score = torch.matmul(q.float().view(b, hkv, -1, d), rows(s["k_cache"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    score = torch.where(live, score, -float("inf"))
    e = torch.exp(score - score.amax(-1, keepdim=True))
    out = torch.matmul(e, rows(s["v_cache"], s["v_scale"])) / e.sum(-1, keepdim=True)
    s["out"].copy_(out.view(b, hq, d))
    return {"out": s["out"]}


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": exact_rotate, "bounds": exact_bounds, "select": lambda s: None, "sparse": exact_sparse}[case["op"]](s)


def exact_rotate(s):
    case, pairs = s["case"], s["case"]["rot"] // 2
    t = s["q"].shape[0]
    pos = s["positions"].view(case["axes"], t)
    table = s["cos_sin"].double()
    turn = torch.empty(t, pairs, dtype=torch.complex128, device=DEVICE)
    a = 0
    for axis, n in enumerate(s["sections"] or [pairs]):
        turn[:, a:a + n] = torch.complex(table[pos[axis]][:, a:a + n], table[pos[axis]][:, pairs + a:pairs + a + n])
        a += n

    def turned(x, w):
        y = x.double().clone()
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * w.double()
        first, second = (slice(0, pairs), slice(pairs, 2 * pairs)) if case["style"] == "halves" else (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2))
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    live = torch.nonzero(s["slot_mapping"] >= 0)[:, 0]
    q = s["q_out"].double()
    q[live] = turned(s["q"], s["q_weight"])[live]
    got = {"q": q}
    for name, rows in (("k", turned(s["key"], s["k_weight"])), ("v", s["value"].double())):
        cache = s[name + "_cache"].double().transpose(1, 2).contiguous()  # [blocks, tokens, heads, dim]
        flat = cache.view(-1, *cache.shape[2:])
        x = rows[live] / s[name + "_scale"]
        flat[s["slot_mapping"][live]] = x.clamp(-448, 448) if s["fp8"] else x
        got[name + "_cache"] = cache.transpose(1, 2).contiguous()
    return got


def exact_bounds(s):
    got, bs = s["key_bounds"].double(), s["block_size"]
    lens, table, new = s["context_lens"].tolist(), s["block_tables"].tolist(), s["new"].tolist()
    ids = torch.tensor([table[b][j] for b, n in enumerate(lens) for j in range((n - new[b]) // bs, n // bs)], dtype=torch.long, device=DEVICE)
    for a in range(0, ids.numel(), 1024):
        i = ids[a:a + 1024]
        k = bits(s["k_cache"])[i].view(s["k_cache"].dtype).double().sort(dim=2).values
        got[i] = torch.stack([k[:, :, 0], k[:, :, -1]], 2)
    return {"key_bounds": got}


def exact_sparse(s):
    case, bs, d, hkv = s["case"], s["block_size"], s["case"]["dim"], s["case"]["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    group = case["q_heads"] // hkv
    kc, vc = bits(s["k_cache"]), bits(s["v_cache"])
    lens = s["context_lens"].tolist()
    chosen = s["selected"].tolist()
    for b, n in enumerate(lens):
        ids = torch.tensor([[j for j in row if j >= 0] for row in chosen[b]], device=DEVICE)  # equally many for each head
        for h in range(hkv):
            phys = s["block_tables"][b][ids[h]].long()
            live = (ids[h][:, None] * bs + torch.arange(bs, device=DEVICE)).view(-1) < n
            k = kc[phys, h].view(s["k_cache"].dtype).view(-1, d)[:live.numel()].double()[live] * s["k_scale"]
            v = vc[phys, h].view(s["v_cache"].dtype).view(-1, d).double()[live] * s["v_scale"]
            p = torch.softmax(s["q"][b, h * group:(h + 1) * group].double() @ k.T * s["scale"], -1)
            out[b, h * group:(h + 1) * group] = p @ v
    return {"out": out}
