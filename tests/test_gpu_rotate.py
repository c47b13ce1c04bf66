"""The rotary append on the GPU against the binary64 definition: norms, both pairings, position axes, 16-bit, f32 and
fp8 caches, fused and unaligned inputs, padding, and what a bad slot or position leaves alone."""
import pytest
import torch

import oracle
import paged_kv_cache_185_gb300 as wllm
from oracle import sparse as S
from tests import sparse_helpers as H

pytestmark = pytest.mark.gpu
BF, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
K_SCALE, V_SCALE = 0.03125, 0.02


def make(T, Hq, Hkv, D, R, bs, dtype, cache, axes=1, weights=None, seed=0, positions=500, shift=0, pad=0, index=torch.int64):
    """Host inputs: q, key and value as slices of one fused tensor whose rows start `shift` elements in."""
    g = H.gen(seed + 31 * T + D + R)
    wide = H.randn(g, T, (Hq + 2 * Hkv) * D + 2 * shift, dtype=dtype)
    fused = wide[:, shift:shift + (Hq + 2 * Hkv) * D]
    blocks = -(-T // bs) + 2
    slots = torch.randperm(blocks * bs, generator=g)[:T].to(index)
    if pad:
        slots[torch.randperm(T, generator=g)[:pad]] = -1
    pos = torch.randint(0, positions, (T,) if axes == 1 else (axes, T), generator=g).to(index)
    w = [None, None] if weights is None else [(1 + H.randn(g, D, scale=0.3)).to(weights) for _ in range(2)]
    pools = [H.cache(g, blocks, Hkv, bs, D, cache) for _ in range(2)]
    return dict(fused=wide, shift=shift, heads=(Hq, Hkv, D), slots=slots, pos=pos, table=H.rotary_table(positions, R),
                q_weight=w[0], k_weight=w[1], kc=pools[0], vc=pools[1], q_out=H.randn(g, T, Hq, D, dtype=dtype))


def parts(x, a):
    Hq, Hkv, D = a["heads"]
    T, at = x.shape[0], a["shift"]
    cut = lambda i, n: x[:, at + i * D:at + (i + n) * D].view(T, n, D) if at == 0 else x[:, at + i * D:at + (i + n) * D].unflatten(1, (n, D))  # noqa: E731
    return cut(0, Hq), cut(Hq, Hkv), cut(Hq + Hkv, Hkv)


def call(a, eps=1e-6, style="halves", sections=None, in_place=False):
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    q, k, v = parts(d["fused"], a)
    out = q if in_place else d["q_out"]
    args = (out, q, k, v, d["kc"], d["vc"], d["slots"], d["pos"], d["table"])
    how = dict(q_weight=d["q_weight"], k_weight=d["k_weight"], eps=eps, style=style, sections=sections)
    if a["kc"].dtype == U8:
        got = wllm.rotate_and_cache_fp8(*args, K_SCALE, V_SCALE, **how)
    else:
        got = wllm.rotate_and_cache(*args, **how)
    assert got is out
    torch.cuda.synchronize()
    return out.cpu(), d["kc"].cpu(), d["vc"].cpu()


def check(a, got, eps=1e-6, style="halves", sections=None, skipped=(), q_before=None, what=""):
    q_out, kc, vc = got
    q, k, v = (x.contiguous() for x in parts(a["fused"], a))
    dtype, fp8, bs = q.dtype, a["kc"].dtype == U8, a["kc"].shape[2]
    live = a["slots"] >= 0
    live[list(skipped)] = False
    ok = lambda x: (x.view(-1, x.shape[-1])[:, live] if x.dim() > 1 else x[live]).clamp(0, a["table"].shape[0] - 1)  # noqa: E731
    pos = ok(a["pos"])
    old = a["q_out"] if q_before is None else q_before
    assert torch.equal(H.bits(q_out.contiguous())[~live], H.bits(old.contiguous())[~live]), f"{what}: q_out of padding"
    ref, size = S.rotate_rows(q[live], pos, a["table"], a["q_weight"], eps, style, sections)
    H.assert_turned(q_out[live], ref, size, dtype, f"{what} q")
    ref, size = S.rotate_rows(k[live], pos, a["table"], a["k_weight"], eps, style, sections)
    slots = a["slots"][live].long()
    rows = lambda c: c[slots // bs, :, slots % bs]  # noqa: E731
    if fp8:
        H.assert_codes(rows(kc), ref / K_SCALE, size / K_SCALE, f"{what} k")
        inv = torch.tensor(oracle.inv_scale(V_SCALE), dtype=F32)
        assert torch.equal(rows(vc), oracle.e4m3_encode(v[live].float() * inv)), f"{what} v"
    else:
        H.assert_turned(rows(kc), ref, size, dtype, f"{what} k")
        assert torch.equal(H.bits(rows(vc)), H.bits(v[live])), f"{what} v"
    rest = torch.ones(kc.shape[0], bs, dtype=torch.bool)
    rest[slots // bs, slots % bs] = False
    for new, was in ((kc, a["kc"]), (vc, a["vc"])):
        assert torch.equal(H.bits(new).transpose(1, 2)[rest], H.bits(was).transpose(1, 2)[rest]), f"{what}: another slot"


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (F16, F16), (F32, F32), (BF, U8), (F16, U8), (F32, U8)])
@pytest.mark.parametrize("style", ["halves", "adjacent"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,bs,weights", [
    (1, 32, 8, 128, 128, 16, True), (37, 28, 4, 128, 64, 16, True), (64, 8, 1, 256, 256, 32, False),
    (5, 3, 3, 64, 32, 8, True), (9, 5, 5, 80, 32, 16, True), (130, 4, 2, 192, 16, 256, False), (700, 7, 1, 16, 16, 1, True)])
def test_rotate_matches_binary64(dtype, cache, style, T, Hq, Hkv, D, R, bs, weights):
    a = make(T, Hq, Hkv, D, R, bs, dtype, cache, weights=dtype if weights else None)
    check(a, call(a, style=style), style=style)


@pytest.mark.parametrize("sections,R", [((16, 24, 24), 128), ((3, 5, 24), 64), ((0, 32), 64), ((8, 8, 8, 8), 64), ((32,), 64)])
@pytest.mark.parametrize("style", ["halves", "adjacent"])
def test_rotate_axes(sections, R, style):
    a = make(50, 8, 2, 128, R, 16, BF, BF, axes=len(sections), weights=F32, seed=2)
    check(a, call(a, style=style, sections=sections), style=style, sections=sections)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (F32, F32), (F16, U8)])
def test_rotate_rows_without_vector_alignment(dtype, cache):
    for shift in (1, 3, 8):
        a = make(33, 6, 2, 128, 128, 16, dtype, cache, weights=dtype, shift=shift, index=torch.int32)
        check(a, call(a), what=f"shift {shift}")
    a = make(33, 6, 2, 128, 48, 16, dtype, cache, weights=dtype)
    wide = torch.zeros(a["table"].shape[0], 51)
    wide[:, 1:49] = a["table"]
    b = dict(a, table=wide)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in b.items()}
    d["table"] = d["table"][:, 1:49]
    q, k, v = parts(d["fused"], a)
    off = torch.zeros(129, dtype=dtype, device="cuda")
    off[1:] = d["k_weight"]
    f, tail = (wllm.rotate_and_cache_fp8, (K_SCALE, V_SCALE)) if cache == U8 else (wllm.rotate_and_cache, ())
    f(d["q_out"], q, k, v, d["kc"], d["vc"], d["slots"], d["pos"], d["table"], *tail, q_weight=d["q_weight"], k_weight=off[1:])
    torch.cuda.synchronize()
    check(a, (d["q_out"].cpu(), d["kc"].cpu(), d["vc"].cpu()), what="table and weight off alignment")


def test_rotate_in_place_padding_and_one_weight():
    a = make(41, 8, 2, 128, 128, 16, BF, BF, weights=BF, pad=6, index=torch.int32)
    before = parts(a["fused"], a)[0].clone()
    check(a, call(a, in_place=True), q_before=before, what="in place")
    for name in ("q_weight", "k_weight"):
        b = dict(a, **{name: None})
        check(b, call(b, eps=0.5), eps=0.5, what=f"without {name}")
    none = dict(a, slots=torch.full_like(a["slots"], -1))
    check(none, call(none), what="all padding")


def test_rotate_many_tokens_and_single_heads():
    check_a = make(6000, 4, 1, 64, 64, 64, F16, F16, weights=F16)
    check(check_a, call(check_a), what="6000 tokens")
    a = make(20, 0, 2, 128, 128, 16, BF, BF)  # keys alone
    check(a, call(a), what="no query heads")


@pytest.mark.parametrize("dtype,cache,Hq,Hkv,D,R,style,sections,weights", [
    (BF, BF, 28, 4, 128, 128, "halves", (16, 24, 24), BF), (F16, U8, 32, 8, 128, 64, "adjacent", None, None),
    (F32, F32, 3, 1, 80, 32, "halves", None, F32), (F32, U8, 8, 8, 64, 64, "adjacent", (5, 27), F32),
    (BF, BF, 5, 5, 256, 256, "halves", None, F32), (F16, F16, 1, 2, 16, 16, "adjacent", None, F16),
    (BF, BF, 64, 64, 256, 256, "halves", None, BF), (BF, U8, 0, 4, 128, 128, "halves", None, BF)])
def test_rotate_a_thousand_tokens(dtype, cache, Hq, Hkv, D, R, style, sections, weights):
    """Enough tokens for the resident form (the 64-head case's tokens are too large for it), with padding among them."""
    a = make(2100 if Hq < 64 else 1100, Hq, Hkv, D, R, 16, dtype, cache, axes=len(sections) if sections else 1, weights=weights, pad=37)
    check(a, call(a, style=style, sections=sections), style=style, sections=sections)
    assert wllm.device_errors() == 0


@pytest.mark.parametrize("T,Hq,Hkv,D,dtype,cache", [
    (270, 28, 4, 128, BF, BF), (271, 28, 4, 128, BF, BF), (410, 32, 8, 64, F16, U8), (160, 32, 16, 128, F32, F32),
    (1220, 4, 1, 128, BF, BF), (151, 128, 8, 128, F16, F16), (153, 128, 8, 128, F16, F16), (300, 16, 16, 80, F32, U8)])
def test_rotate_where_the_resident_form_begins(T, Hq, Hkv, D, dtype, cache):
    """Token counts about the first that the resident form takes, with norms whose weights are binary32."""
    a = make(T, Hq, Hkv, D, D // 32 * 16, 16, dtype, cache, weights=F32, seed=5)
    check(a, call(a))


def test_rotate_a_thousand_tokens_strided_in_place_and_bad():
    T, Hq, Hkv, D = 1500, 6, 2, 64
    a = make(T, Hq, Hkv, D, 64, 16, BF, BF, weights=BF, pad=20, index=torch.int32)
    live = (a["slots"] >= 0).nonzero()[:, 0]
    a["slots"][live[5]], a["pos"][live[400]], a["pos"][live[-1]] = 10 ** 6, 500, -3
    skipped = live[[5, 400, -1]].tolist()
    before = parts(a["fused"], a)[0].clone()
    got = call(a, in_place=True)
    assert wllm.device_errors() == 1 | 32
    check(a, got, skipped=skipped, q_before=before, what="in place")
    # heads that do not lie next to each other
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    wide = [torch.zeros(T, n, D + 8, dtype=BF, device="cuda") for n in (Hq, Hkv, Hkv)]
    for w, x in zip(wide, parts(d["fused"], a)):
        w[:, :, :D] = x
    q, k, v = (w[:, :, :D] for w in wide)
    out = torch.zeros(T, Hq, D + 16, dtype=BF, device="cuda")
    out[:, :, 8:D + 8] = d["q_out"]
    wllm.rotate_and_cache(out[:, :, 8:D + 8], q, k, v, d["kc"], d["vc"], d["slots"], d["pos"], d["table"],
                          q_weight=d["q_weight"], k_weight=d["k_weight"])
    torch.cuda.synchronize()
    assert wllm.device_errors() == 1 | 32
    check(a, (out[:, :, 8:D + 8].cpu(), d["kc"].cpu(), d["vc"].cpu()), skipped=skipped, what="strided")
    assert (out[:, :, :8] == 0).all() and (out[:, :, D + 8:] == 0).all()


def test_rotate_leaves_out_tokens_with_a_bad_slot_or_position(monkeypatch):
    assert wllm.device_errors() == 0
    a = make(24, 4, 2, 64, 64, 16, BF, BF, weights=BF)
    a["slots"][3] = a["kc"].shape[0] * 16
    a["pos"][7], a["pos"][9] = 500, -1
    got = call(a)
    assert wllm.device_errors() == 1 | 32
    check(a, got, skipped=(3, 7, 9), what="bad")
    monkeypatch.setenv("WLLM_CHECK", "1")
    with pytest.raises(wllm.WllmError, match="0x1\\b"):
        call(a)
    a["slots"][3] = -1
    with pytest.raises(wllm.WllmError, match="0x20"):
        call(a)
    a["pos"][7] = a["pos"][9] = 0
    call(a)
    assert wllm.device_errors() == 0


def test_rotate_extreme_rows():
    """Zero rows stay zero under the norm, huge ones saturate E4M3 at 448 and NaN stays NaN."""
    a = make(4, 1, 1, 64, 64, 16, F32, U8, weights=F32)
    a["fused"][0] = 0.0
    a["fused"][1] = 1e5
    a["fused"][2] = float("nan")
    a["pos"][:] = 0
    a["k_weight"] = None
    q, kc, vc = call(a)
    at = lambda c, t: oracle.widen_e4m3(c[a["slots"][t] // 16, :, a["slots"][t] % 16])  # noqa: E731
    assert (q[0] == 0).all() and (at(kc, 0) == 0).all()
    assert (at(kc, 1) == 448).all() and (at(vc, 1) == 448).all()
    assert q[2].isnan().all() and at(kc, 2).isnan().all() and at(vc, 2).isnan().all()


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (F16, F16), (F32, F32), (F16, U8)])
@pytest.mark.parametrize("style", ["halves", "adjacent"])
@pytest.mark.parametrize("T,Hq,D,R,shift", [(5, 4, 128, 32, 0), (5, 4, 128, 64, 1), (9, 3, 80, 16, 0), (2000, 4, 64, 32, 0), (2000, 4, 128, 32, 0)])
def test_rotate_leaves_the_elements_behind_the_turned_ones_alone(dtype, cache, style, T, Hq, D, R, shift):
    """Without a norm the elements from R on come out as they went in (as codes: of their own value), whatever their
    neighbours hold: infinities and NaN do not spread, and a zero keeps its sign.  (A NaN is any NaN: rounding to the 16-bit
    type does not keep its payload.)"""
    a = make(T, Hq, 2, D, R, 16, dtype, cache, shift=shift, seed=9)
    q, k, _ = parts(a["fused"], a)
    for x in (q, k):
        x[..., R] = float("inf")
        x[..., R + 3] = float("nan")
        x[..., D - 5] = -float("inf")
        x[..., R + 1], x[..., R + 6], x[..., D - 2], x[..., D - 9] = -0.0, 0.0, -0.0, -0.0
    same = lambda x, y: bool(((H.bits(x.contiguous()) == H.bits(y.contiguous())) | (x.isnan() & y.isnan())).all())  # noqa: E731
    q_out, kc, _ = call(a, style=style)
    assert same(q_out[..., R:], q[..., R:])
    slots = a["slots"].long()
    got = kc[slots // 16, :, slots % 16][..., R:].contiguous()
    if cache == U8:
        inv = torch.tensor(oracle.inv_scale(K_SCALE), dtype=F32)
        assert torch.equal(got, oracle.e4m3_encode(k[..., R:].float() * inv))
    else:
        assert same(got, k[..., R:])


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("style", ["halves", "adjacent"])
@pytest.mark.parametrize("T,D,R", [(6, 128, 32), (2000, 64, 32)])
def test_rotate_norms_an_infinite_row_element_by_element(dtype, cache, style, T, D, R):
    """x / sqrt(inf) is zero for the finite elements behind the turned ones and NaN for the infinite one alone."""
    a = make(T, 4, 2, D, R, 16, dtype, cache, weights=dtype, seed=10)
    q, k, _ = parts(a["fused"], a)
    for x in (q, k):
        x[..., R + 2] = float("inf")
    q_out, kc, _ = call(a, style=style)
    slots = a["slots"].long()
    for got in (q_out, kc[slots // 16, :, slots % 16]):
        want = torch.zeros_like(got[..., R:])
        want[..., 2] = float("nan")
        assert torch.equal(got[..., R:].nan_to_num(7.0), want.nan_to_num(7.0))
