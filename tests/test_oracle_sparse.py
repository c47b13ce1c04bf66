"""The binary64 definitions of the rotary append and block-sparse decode against brute force and invariants."""
import math

import pytest
import torch

import oracle
from oracle import sparse as S
from tests import sparse_helpers as H


@pytest.mark.parametrize("style", ["halves", "adjacent"])
def test_turn_keeps_lengths_and_depends_on_distance_only(style):
    g = H.gen(1)
    table = H.rotary_table(64, 32)
    x = H.randn(g, 2, 1, 32, dtype=torch.float64).float()

    def dot(i, j):
        a, _ = S.rotate_rows(x[:1], torch.tensor([i]), table, style=style)
        b, _ = S.rotate_rows(x[1:], torch.tensor([j]), table, style=style)
        return (a * b).sum().item()

    y, size = S.rotate_rows(x, torch.tensor([3, 60]), table, style=style)
    assert torch.allclose(y.pow(2).sum(-1), x.double().pow(2).sum(-1), rtol=1e-6)
    assert torch.allclose(size.pow(2).sum(-1), 2 * x.double().pow(2).sum(-1), rtol=1e-12)
    assert abs(dot(5, 9) - dot(40, 44)) < 1e-5 and abs(dot(5, 9) - dot(9, 5)) > 1e-3


def test_axes_turn_their_own_pairs():
    g = H.gen(2)
    x = H.randn(g, 3, 2, 64)
    table = H.rotary_table(50, 48)
    pos = torch.tensor([[1, 2, 3], [10, 20, 30], [0, 0, 0]])
    y, _ = S.rotate_rows(x, pos, table, sections=[4, 8, 12])
    for axis, (a, b) in enumerate([(0, 4), (4, 12), (12, 24)]):
        alone, _ = S.rotate_rows(x, pos[axis], table)
        assert torch.equal(y[..., a:b], alone[..., a:b]) and torch.equal(y[..., 24 + a:24 + b], alone[..., 24 + a:24 + b])
    assert torch.equal(y[..., 48:], x[..., 48:].double())  # behind the turned part
    assert torch.equal(y[..., 12:24], x[..., 12:24].double())  # position 0


def test_norm_gives_rows_of_unit_mean_square():
    x = H.randn(H.gen(3), 4, 3, 32, scale=7.0)
    y, _ = S.rotate_rows(x, torch.zeros(4, dtype=torch.long), H.rotary_table(1, 16), weight=torch.ones(32), eps=0.0)
    assert torch.allclose(y.pow(2).mean(-1), torch.ones(4, 3, dtype=torch.float64), rtol=1e-12)


def test_scores_bound_every_key():
    g = H.gen(4)
    bt, pool = H.block_tables(g, [100], 16)
    k = H.randn(g, pool, 2, 16, 32)
    q = H.randn(g, 1, 6, 32)
    bounds = S.key_bounds(k, bt, torch.tensor([112]), [112], torch.zeros(pool, 2, 2, 32, dtype=torch.float64)).float()
    s = S.scores(q, bounds, bt, torch.tensor([100]), 2, 16)[0]
    for h in range(2):
        for j in range(7):
            dots = k[bt[0, j], h].double() @ q[0, 3 * h:3 * h + 3].double().T
            assert (dots.amax(0).sum() <= s[h, j] + 1e-9)


def test_selection_of_everything_is_the_decode():
    g = H.gen(5)
    lens = [1, 40, 77, 0]
    bt, pool = H.block_tables(g, lens, 16)
    kc, vc = H.cache(g, pool, 2, 16, 64, torch.float32), H.cache(g, pool, 2, 16, 64, torch.float32)
    q = H.randn(g, 4, 4, 64)
    cl = torch.tensor(lens, dtype=torch.int32)
    bounds = torch.zeros(pool, 2, 2, 64)
    sel = S.select_blocks(q, bounds, bt, cl, 2, 16, 5, 0, 1)
    assert sel[2, 0].tolist() == [0, 1, 2, 3, 4] and sel[1, 1].tolist() == [0, 1, 2, -1, -1] and sel[3, 0].tolist() == [-1] * 5
    scale = 1 / math.sqrt(64)
    out, mag, _ = S.sparse_decode(q, kc, vc, bt, cl, sel, scale)
    ref = oracle.paged_decode(q, kc, vc, bt, cl, 2, scale)
    assert torch.allclose(out, ref, atol=1e-6) and (mag >= out.abs() - 1e-12).all()


def test_ties_and_nan_in_the_selection():
    lens = [16 * 8]
    bt = torch.arange(8, dtype=torch.int32)[None]
    bounds = torch.ones(8, 1, 2, 64)
    bounds[5] = float("nan")
    q = torch.ones(1, 2, 64)
    sel = S.select_blocks(q, bounds, bt, torch.tensor(lens), 1, 16, 4, 1, 1)
    assert sel[0, 0].tolist() == [0, 1, 5, 7]  # the first, the lowest of the equal, the NaN, the last
