"""Cases that measure a paged cache of 8-bit codes with a scale for each block and head, from the blocks' allocation to
the attention that reads it.

Four operators make one step of a server that keeps its lengths, tables and free blocks on the GPU:

  slots    assign_slots: blocks taken from (and given back to) a list of free ones, table entries, slots, positions and
           packed starts of the tokens that each sequence is to get
  append   reshape_and_cache_block_scaled: new keys and values stored as E4M3 codes under their block's and head's scale,
           a power of two, which rises where the new ones need it (the block's earlier codes are stored again then)
  decode   paged_attention_decode_block_scaled: one query token per sequence
  prefill  paged_attention_prefill_block_scaled: packed chunks of query tokens, causal

``run`` with ``own`` false is the plain form in elementary torch operations; with ``own`` true it is the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
F8 = torch.float8_e4m3fn
DEVICE = "cuda"
MOST = 448.0            # the largest E4M3 value
LEAST_E, MOST_E = -40, 40  # exponents of the scales


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a small server: the call's own latency
        dict(name="slots step of 32", op="slots", seqs=32, prompts=0, ended=0, lo=100, hi=4000, chunk=0, rows=32, block=16),
        # a busy server's step: decodes, chunks of prompts among them, some sequences that have ended; rows padded
        dict(name="slots mixed 512", op="slots", seqs=512, prompts=8, ended=24, lo=100, hi=8000, chunk=900, rows=8192, block=16),
        # prompts only, as a batch job begins
        dict(name="slots prompts 64K", op="slots", seqs=40, prompts=40, ended=0, lo=0, hi=0, chunk=1600, rows=65536, block=32),
        # one decode step of a few interactive requests: the call's own latency
        dict(name="append step of 8", op="append", seqs=8, lo=100, hi=4000, chunk=1, empty=0, kv_heads=8, dim=128, block=16,
             dtype="bf16"),
        # one decode step of a full batch, padded to its captured size with empty sequences
        dict(name="append step of 256", op="append", seqs=256, lo=100, hi=4000, chunk=1, empty=5, kv_heads=4, dim=128, block=16,
             dtype="bf16"),
        # chunks of prompts, most of them continued inside a block
        dict(name="append prompts", op="append", seqs=16, lo=1100, hi=6000, chunk=1024, empty=0, kv_heads=8, dim=128, block=16,
             dtype="bf16"),
        # a single long chat
        dict(name="decode one 16K", op="decode", seqs=1, lo=16000, hi=16000, q_heads=32, kv_heads=4, dim=64, block=16, dtype="f16"),
        # long documents
        dict(name="decode 8 long", op="decode", seqs=8, lo=32768, hi=131072, q_heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16"),
        # a busy server
        dict(name="decode 256", op="decode", seqs=256, lo=300, hi=6000, q_heads=28, kv_heads=4, dim=128, block=16, dtype="bf16"),
        # the next turn of one chat
        dict(name="prefill one turn", op="prefill", seqs=1, lo=2100, hi=2100, chunk=100, q_heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16"),
        # a few drafted tokens of every sequence, to be checked together
        dict(name="prefill drafts", op="prefill", seqs=64, lo=300, hi=6000, chunk=5, q_heads=28, kv_heads=4, dim=128, block=16,
             dtype="bf16"),
        # chunks of long prompts
        dict(name="prefill prompts", op="prefill", seqs=8, lo=1024, hi=6144, chunk=1024, q_heads=28, kv_heads=4, dim=128, block=16,
             dtype="bf16"),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["slots", "append", "decode", "prefill"])
    block = rng.choice([8, 16, 16, 32, 64])
    if op == "slots":
        seqs = spread(rng, 1, 1500)
        prompts = min(seqs, rng.choice([0, spread(rng, 1, 40), spread(rng, 1, 40)]))
        hi = spread(rng, 1, 20000)
        chunk = spread(rng, 1, 1600)
        rows = min(65536, seqs + prompts * chunk + rng.choice([0, 0, 7, 500]))
        return dict(op=op, seqs=seqs, prompts=prompts, ended=rng.choice([0, seqs // 12]), lo=rng.randint(0, hi), hi=hi, chunk=chunk,
                    rows=rows, block=block)
    group, kv_heads = rng.choice([(1, 8), (1, 32), (4, 8), (7, 4), (8, 4), (8, 1), (16, 2), (5, 2), (3, 5)])
    dim = rng.choice([64, 128, 128, 256])
    row = kv_heads * dim
    if op == "append":
        dtype = rng.choice(["bf16", "f16", "bf16", "f32"])
        chunk = rng.choice([1, spread(rng, 2, 2048)])
        seqs = max(1, min(spread(rng, 1, 300), int(3.3e7 / (chunk * row * BYTES[dtype]))))
        lo = spread(rng, 1, 4000)
        hi = max(lo, min(spread(rng, lo, 20000), int(2e8 / (seqs * row))))
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, chunk=chunk, empty=rng.choice([0, 0, 3]), kv_heads=kv_heads, dim=dim, block=block,
                    dtype=dtype)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "prefill":
        dim = min(dim, 128)
        row = kv_heads * dim
    if dim == 64:
        block = max(block, 16)
    case = dict(op=op, seqs=0, lo=0, hi=0, q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim, block=block, dtype=dtype)
    if op == "decode":
        seqs = spread(rng, 1, 256)
        hi = max(1, min(spread(rng, 1, 131072), int(6e8 / (row * seqs))))
        case.update(seqs=seqs, lo=rng.choice([1, rng.randint(1, hi), hi]), hi=hi)
        return case
    chunk = spread(rng, 1, 2048)
    seqs = spread(rng, 1, 64)
    hi = chunk + spread(rng, 1, 8192) - 1
    seqs = max(1, min(seqs, int(1.3e9 / (case["q_heads"] * chunk * hi)), int(4e8 / (row * hi))))
    hi = min(hi, max(chunk, int(1.3e9 / (case["q_heads"] * chunk * seqs))))
    case.update(seqs=seqs, lo=rng.randint(1, hi), hi=hi, chunk=chunk)
    return case


# ---------------------------------------------------------------- sizes that follow from a case alone
def ragged(count, lo, hi):
    """`count` lengths spread evenly over lo..hi, in an order without pattern."""
    return [lo + int((hi - lo + 1) * ((0.5 + 0.6180339887498949 * i) % 1.0)) for i in range(count)]


def chunk_of(i, n, chunk):
    """New tokens of the sequence at place i that has n tokens with them: about `chunk`, of uneven number."""
    return min(n, chunk if chunk <= 8 else max(1, chunk - (37 * i) % (chunk // 3 + 1)))


def requests(case):
    """(tokens held, tokens to add; -1 for one that has ended) of the sequences of a slots case."""
    lens = ragged(case["seqs"], case["lo"], case["hi"])
    new = [1] * case["seqs"]
    for i in range(case["prompts"]):
        new[i * case["seqs"] // case["prompts"]] = chunk_of(i, 1 << 30, case["chunk"])
    for i in range(case["ended"]):
        new[(i * 12 + 5) % case["seqs"]] = -1
    return lens, new


def work(case):
    bs = case["block"]
    if case["op"] == "slots":
        lens, new = requests(case)
        blocks = sum(-(-(n + max(m, 0)) // bs) - -(-n // bs) if m >= 0 else -(-n // bs) for n, m in zip(lens, new))
        # lengths, wishes, starts; entries moved between list and tables; slots and positions
        return {"bytes": case["seqs"] * 16 + blocks * 8 + case["rows"] * 16 + 8, "flops": 0}
    hkv, d = case["kv_heads"], case["dim"]
    lens = ragged(case["seqs"], case["lo"], case["hi"])
    blocks = sum(-(-n // bs) for n in lens)
    if case["op"] == "append":
        new = [chunk_of(i, n, case["chunk"]) for i, n in enumerate(lens)]
        touched = sum(-(-n // bs) - (n - m) // bs for n, m in zip(lens, new))
        values = sum(new) * hkv * 2 * d
        return {"bytes": values * (BYTES[case["dtype"]] + 1) + touched * (hkv * 2 * 8 + 4) + 8 * len(lens), "flops": 2 * values}
    hq, e, tokens = case["q_heads"], BYTES[case["dtype"]], sum(lens)
    held = tokens * hkv * 2 * d + blocks * (hkv * 2 * 4 + 4) + 4 * len(lens)
    if case["op"] == "decode":
        return {"bytes": held + 2 * len(lens) * hq * d * e, "flops": tokens * hq * d * 4}
    new = [chunk_of(i, n, case["chunk"]) for i, n in enumerate(lens)]
    pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new))
    return {"bytes": held + 2 * sum(new) * hq * d * e + 4 * len(lens), "flops": pairs * hq * d * 4}


# ---------------------------------------------------------------- inputs
def tables(gen, counts, width):
    """Block tables for sequences of `counts` blocks out of a shuffled pool (-1 past a sequence's last), and the free blocks."""
    used = sum(counts)
    order = torch.randperm(used + 3, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEVICE)
    at = torch.arange(width, device=DEVICE)[None, :]
    table[at < torch.tensor(counts, device=DEVICE)[:, None]] = order[:used]
    return table, order[used:]


def pool(gen, shape, keys):
    """Codes and scales of a cache as it comes: keys have a bias for each channel, blocks and heads differ in size; [blocks, heads, tokens, dim]."""
    n, h, bs, d = shape
    codes = torch.empty(shape, dtype=F8, device=DEVICE)
    scales = torch.empty(n, h, dtype=torch.float32, device=DEVICE)
    bias = torch.randn(h, 1, d, generator=gen, device=DEVICE) if keys else 0.0
    for a in range(0, n, 4096):
        m = min(4096, n - a)
        size = torch.exp(0.4 * torch.randn(m, h, 1, 1, generator=gen, device=DEVICE))
        x = (torch.randn(m, h, bs, d, generator=gen, device=DEVICE) + bias) * size
        e = torch.ceil(torch.log2(x.abs().amax((2, 3)).double() / MOST))
        scales[a:a + m] = torch.exp2(e).float()
        codes[a:a + m] = (x / scales[a:a + m, :, None, None]).to(F8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    s = {"case": case, "block_size": case["block"]}
    if case["op"] == "slots":
        return prepare_slots(s, case, gen)
    d, bs, hkv, dt = case["dim"], case["block"], case["kv_heads"], DTYPES[case["dtype"]]
    lens = ragged(case["seqs"], case["lo"], case["hi"])
    new = [chunk_of(i, n, case.get("chunk", 1)) for i, n in enumerate(lens)]
    order = torch.randperm(len(lens), generator=gen, device=DEVICE).tolist()
    lens, new = [lens[i] for i in order] + [0] * case.get("empty", 0), [new[i] for i in order] + [0] * case.get("empty", 0)
    blocks = [-(-n // bs) for n in lens]
    s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    s["block_tables"], spare = tables(gen, blocks, max(blocks))
    shape = (sum(blocks) + spare.numel(), hkv, bs, d)
    s["k_cache"], s["k_scales"] = pool(gen, shape, True)
    s["v_cache"], s["v_scales"] = pool(gen, shape, False)
    single = case["op"] == "decode" or case["op"] == "append" and case["chunk"] == 1
    starts = torch.tensor([0] + new, device=DEVICE).cumsum(0).to(torch.int32)
    s["query_start_loc"] = None if single else starts
    rows = len(lens) if single else sum(new)
    s["rows"] = rows
    if case["op"] == "append":
        # slices of a fused projection's output; sizes differ from token to token
        fused = torch.randn(rows, 2 * hkv * d, generator=gen, device=DEVICE)
        fused = (fused * torch.exp(0.4 * torch.randn(rows, 1, generator=gen, device=DEVICE))).to(dt)
        s["key"] = fused[:, :hkv * d].view(rows, hkv, d)
        s["value"] = fused[:, hkv * d:].view(rows, hkv, d)
        return s
    s["q"] = torch.randn(rows, case["q_heads"], d, generator=gen, device=DEVICE).to(dt)
    s["out"] = torch.empty_like(s["q"])
    s["scale"] = 1.0 / math.sqrt(d)
    s["longest"], s["most_new"] = max(lens), max(new)
    return s


def prepare_slots(s, case, gen):
    bs = case["block"]
    lens, new = requests(case)
    order = torch.randperm(len(lens), generator=gen, device=DEVICE).tolist()
    lens, new = [lens[i] for i in order], [new[i] for i in order]
    held = [-(-n // bs) for n in lens]
    need = sum(-(-(n + m) // bs) - h for n, m, h in zip(lens, new, held) if m >= 0)
    width = -(-(max(lens) + max(case["chunk"], 1)) // bs) + 1
    s["block_tables"], _ = tables(gen, held, width)
    # the list has room for the whole pool; every tenth state runs short of blocks at its end
    count = max(0, need - sum(h for h, m in zip(held, new) if m < 0) + (-3 if int(torch.randint(0, 10, (1,), generator=gen, device=DEVICE)) == 0 else 40))
    s["free_blocks"] = torch.full((count + sum(held) + 40,), -1, dtype=torch.int32, device=DEVICE)
    s["free_blocks"][:count] = sum(held) + 3 + torch.randperm(count, generator=gen, device=DEVICE).to(torch.int32)
    s["num_free"] = torch.tensor([count], dtype=torch.int32, device=DEVICE)
    s["context_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    s["new_tokens"] = torch.tensor(new, dtype=torch.int32, device=DEVICE)
    s["slot_mapping"] = torch.empty(case["rows"], dtype=torch.int64, device=DEVICE)
    s["positions"] = torch.empty(case["rows"], dtype=torch.int64, device=DEVICE)
    s["query_start_loc"] = torch.empty(len(lens) + 1, dtype=torch.int32, device=DEVICE)
    s["context_lens_out"] = torch.empty_like(s["context_lens"])
    s["num_free_out"] = torch.empty_like(s["num_free"])
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return (run_own if own else run_plain)(s)


def run_own(s):
    import paged_kv_cache_185_gb300 as wllm
    case, bs = s["case"], s["block_size"]
    if case["op"] == "slots":
        wllm.assign_slots(s["slot_mapping"], s["query_start_loc"], s["block_tables"], s["context_lens"], s["new_tokens"],
                          s["free_blocks"], s["num_free"], bs, positions=s["positions"],
                          context_lens_out=s["context_lens_out"], num_free_out=s["num_free_out"])
        return slots_outputs(s)
    cache = [s[k] for k in ("k_cache", "v_cache", "k_scales", "v_scales", "block_tables", "context_lens")]
    if case["op"] == "append":
        wllm.reshape_and_cache_block_scaled(s["key"], s["value"], *cache, bs, query_start_loc=s["query_start_loc"])
        return append_outputs(s)
    if case["op"] == "decode":
        wllm.paged_attention_decode_block_scaled(s["out"], s["q"], *cache, case["kv_heads"], s["scale"], bs)
    else:
        wllm.paged_attention_prefill_block_scaled(s["out"], s["q"], *cache, s["query_start_loc"], case["kv_heads"], s["scale"], bs)
    return {"out": s["out"]}


def slots_outputs(s):
    return {k: s[k] for k in ("slot_mapping", "positions", "query_start_loc", "context_lens_out", "num_free_out", "block_tables",
                              "free_blocks")}


def append_outputs(s):
    return {k: s[k] for k in ("k_cache", "v_cache", "k_scales", "v_scales")}


def run_plain(s):
    return {"slots": plain_slots, "append": plain_append, "decode": plain_decode, "prefill": plain_prefill}[s["case"]["op"]](s)


def bits(x):
    """The same storage as whole numbers, for indexed reads and writes of codes."""
    return x.view(torch.uint8)


def plain_slots(s):
    bs, table, free = s["block_size"], s["block_tables"], s["free_blocks"]
    lens, new = s["context_lens"].long(), s["new_tokens"].long()
    rows, width = s["slot_mapping"].numel(), table.shape[1]
    held = (lens + bs - 1) // bs
    ended = new < 0
    fits = ~ended & (lens + new <= width * bs)
    want = torch.where(fits, new, 0)
    need = torch.where(fits, (lens + new + bs - 1) // bs - held, 0)
    # blocks of the sequences that have ended come on top of the list, then the new ones are taken from its top
    gone = torch.where(ended, held, 0)
    at = torch.arange(width, device=DEVICE)[None, :]
    back = at < gone[:, None]
    free[(s["num_free"].long() + (gone.cumsum(0) - gone)[:, None] + at)[back]] = table[back]
    count = s["num_free"].long() + gone.sum()
    upto = need.cumsum(0)
    served = fits & (want.cumsum(0) <= rows) & ((need == 0) | (upto <= count))
    k = at - held[:, None]
    taken = served[:, None] & (k >= 0) & (k < need[:, None])
    table[taken] = free[(count - 1 - (upto - need)[:, None] - k)[taken]]
    got = torch.where(served, want, 0)
    starts = torch.cat([got.new_zeros(1), got.cumsum(0)])
    s["query_start_loc"].copy_(starts)
    s["context_lens_out"].copy_(torch.where(ended, 0, lens + got))
    s["num_free_out"].copy_(count - torch.where(served, need, 0).sum())
    t = torch.arange(rows, device=DEVICE)
    seq = torch.searchsorted(starts[1:], t, right=True).clamp(max=lens.numel() - 1)
    pos = lens[seq] + t - starts[seq]
    live = t < starts[-1]
    block = table[seq, torch.where(live, pos // bs, 0)].long()
    s["slot_mapping"].copy_(torch.where(live, block * bs + pos % bs, -1))
    s["positions"].copy_(torch.where(live, pos, 0))
    return slots_outputs(s)


def new_rows(s):
    """(sequence, position) of each packed row, the new tokens of each sequence, and which rows are some sequence's."""
    lens = s["context_lens"].long()
    if s["query_start_loc"] is None:
        return torch.arange(lens.numel(), device=DEVICE), lens - 1, (lens > 0).long(), lens > 0
    starts = s["query_start_loc"].long()
    t = torch.arange(s["rows"], device=DEVICE)
    seq = torch.searchsorted(starts[1:], t, right=True).clamp(max=lens.numel() - 1)
    new = starts[1:] - starts[:-1]
    return seq, (lens - new)[seq] + t - starts[seq], new, t < starts[-1]


def plain_append(s):
    bs, table, lens = s["block_size"], s["block_tables"], s["context_lens"].long()
    seq, pos, new, live = new_rows(s)
    seq, pos = seq[live], pos[live]
    block = table[seq, pos // bs].long()
    # the block in which each sequence's new tokens begin, where it holds earlier ones
    first = lens - new
    open_ = (new > 0) & (first % bs > 0)
    old_block = table[torch.arange(lens.numel(), device=DEVICE), torch.where(open_, first // bs, 0)].long()[open_]
    earlier = torch.arange(bs, device=DEVICE)[None, :] < (first % bs)[open_][:, None]
    for name in ("key", "value"):
        cache, scales = s[name[0] + "_cache"], s[name[0] + "_scales"]
        x = s[name][live].float()
        size = x.abs().amax(-1)
        most = torch.zeros_like(scales).index_reduce_(0, block, size, "amax")
        # in 64 bits: a value of exactly 448 2^e takes 2^e
        m, e = torch.frexp(most.double() / MOST)
        e = torch.where(most > 0, e - (m == 0.5).to(e.dtype), LEAST_E).clamp(LEAST_E, MOST_E)
        need = torch.exp2(e.double()).float()
        was = scales.clone()
        touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=DEVICE)
        touched[block] = True
        scales.copy_(torch.where(touched[:, None], need, was))
        scales[old_block] = torch.maximum(was[old_block], need[old_block])
        held = bits(cache)[old_block]  # [n, heads, tokens, dim]
        factor = was[old_block] * (1.0 / scales[old_block])
        again = (held.view(F8).float() * factor[:, :, None, None]).clamp(-MOST, MOST).to(F8)
        bits(cache)[old_block] = torch.where(earlier[:, None, :, None], bits(again), held)
        codes = (x * (1.0 / scales[block])[:, :, None]).clamp(-MOST, MOST).to(F8)
        bits(cache)[block, :, pos % bs] = bits(codes)
    return append_outputs(s)


def dense(s, cache, scales):
    """The cached rows of every sequence, [sequences, heads, tokens, dim] in 32 bits, zero past a sequence's length."""
    bs, lens = s["block_size"], s["context_lens"].long()
    ids = s["block_tables"][:, :-(-s["longest"] // bs)].long().clamp(min=0)
    x = bits(cache)[ids].view(F8).float() * scales[ids][..., None, None]  # [B, blocks, heads, tokens, dim]
    x = x.transpose(1, 2).flatten(2, 3)
    live = torch.arange(x.shape[2], device=DEVICE)[None, :] < lens[:, None]
    return torch.where(live[:, None, :, None], x, 0.0), live


def plain_decode(s):
    q, hkv = s["q"], s["case"]["kv_heads"]
    b, hq, d = q.shape
    k, live = dense(s, s["k_cache"], s["k_scales"])
    score = torch.matmul(q.float().view(b, hkv, hq // hkv, d), k.transpose(2, 3)) * s["scale"]
    del k
    score = torch.where(live[:, None, None, :], score, -float("inf"))
    e = torch.exp(score - score.amax(-1, keepdim=True))
    v, _ = dense(s, s["v_cache"], s["v_scales"])
    s["out"].copy_((torch.matmul(e, v) / e.sum(-1, keepdim=True)).view(b, hq, d))
    return {"out": s["out"]}


def plain_prefill(s):
    q, hkv, most = s["q"], s["case"]["kv_heads"], s["most_new"]
    t, hq, d = q.shape
    seq, pos, new, _ = new_rows(s)
    at = torch.arange(t, device=DEVICE) - s["query_start_loc"].long()[seq]
    b, g = new.numel(), hq // hkv
    padded = torch.zeros(b, most, hq, d, device=DEVICE)
    padded[seq, at] = q.float()
    where = torch.zeros(b, most, dtype=torch.long, device=DEVICE)
    where[seq, at] = pos
    rows = padded.view(b, most, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * most, d)
    k, _ = dense(s, s["k_cache"], s["k_scales"])
    score = torch.matmul(rows, k.transpose(2, 3)).view(b, hkv, g, most, -1) * s["scale"]
    del k
    seen = torch.arange(score.shape[-1], device=DEVICE) <= where[:, None, None, :, None]
    score = torch.where(seen, score, -float("inf"))
    e = torch.exp(score - score.amax(-1, keepdim=True))
    del score, seen
    v, _ = dense(s, s["v_cache"], s["v_scales"])
    out = torch.matmul(e.view(b, hkv, g * most, -1), v).view(b, hkv, g, most, d) / e.sum(-1, keepdim=True)
    s["out"].copy_(out.permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)[seq, at])
    return {"out": s["out"]}


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers only
    if case["op"] != "append" and work(case)["flops"] > 1.5e12:
        return None
    s = prepare(case, seed)
    return exact_append(s) if case["op"] == "append" else exact_attention(s)


def exact_append(s):
    bs, lens, table = s["block_size"], s["context_lens"].tolist(), s["block_tables"].tolist()
    starts = s["query_start_loc"].tolist() if s["query_start_loc"] is not None else None
    got = {}
    for name in ("key", "value"):
        codes, scales = s[name[0] + "_cache"].double(), s[name[0] + "_scales"].double()
        x = s[name].double()
        for b, n in enumerate(lens):
            row, new = (b, min(n, 1)) if starts is None else (starts[b], starts[b + 1] - starts[b])
            at = n - new
            while at < n:
                j, off = at // bs, at % bs
                rows = x[row:row + min(bs - off, n - at)].transpose(0, 1)  # [heads, tokens, dim]
                i = table[b][j]
                size = rows.abs().amax((1, 2)) / 448
                e = torch.floor(torch.log2(size.clamp(min=2.0 ** -60)))
                e = torch.where(torch.exp2(e) < size, e + 1, e).clamp(LEAST_E, MOST_E)
                to = torch.exp2(e)
                if off:
                    to = torch.maximum(to, scales[i])
                    codes[i, :, :off] *= (scales[i] / to)[:, None, None]
                scales[i] = to
                codes[i, :, off:off + rows.shape[1]] = (rows / to[:, None, None]).clamp(-448, 448)
                at, row = at + rows.shape[1], row + rows.shape[1]
        got[name[0] + "_cache"], got[name[0] + "_scales"] = codes, scales
    return got


def exact_attention(s):
    case, bs, d, hkv = s["case"], s["block_size"], s["case"]["dim"], s["case"]["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    group, lens = case["q_heads"] // hkv, s["context_lens"].tolist()
    starts = s["query_start_loc"].tolist() if s["query_start_loc"] is not None else list(range(len(lens) + 1))
    for b, n in enumerate(lens):
        phys = s["block_tables"][b, :-(-n // bs)].long()
        r0, r1 = starts[b], starts[b + 1]
        pos = torch.arange(n - (r1 - r0), n, device=DEVICE)
        for h in range(hkv):
            k, v = (bits(s[x + "_cache"])[phys, h].view(F8).double().mul(s[x + "_scales"][phys, h].double()[:, None, None]).view(-1, d)[:n]
                    for x in "kv")
            for g in range(h * group, (h + 1) * group):
                p = s["q"][r0:r1, g].double() @ k.T * s["scale"]
                p = torch.softmax(p.masked_fill(torch.arange(n, device=DEVICE)[None, :] > pos[:, None], -float("inf")), -1)
                out[r0:r1, g] = p @ v
    return {"out": out}
