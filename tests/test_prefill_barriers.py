"""The warps of the block-scaled prefill and their mbarriers, as a model under random schedules.

A wait on an mbarrier tells two phases apart, by their parity: one that comes a phase too early passes as if its own were
over.  The model has the kernel's agents (two producers, two widening pairs, an MMA warp and the softmax of each of two
streams), its rings and its waits; copies land in any order, and what an MMA warp has issued completes in its order.  Every
wait that passes asserts what it was for, every arrival that it is not one too many.  Ring sizes are the source's."""
import os
import random
import re

import pytest

from paged_kv_cache_185_gb300 import build

SOURCE = open(os.path.join(build.CSRC, "prefill_block_scaled.cu")).read()


def constant(name):
    return int(re.search(rf"\b{name} = (\d+)\b", SOURCE).group(1))


SLOTS, MORE_SLOTS, RAWS, FACTORS = (constant(n) for n in ("kSlots", "kMoreSlots", "kRaws", "kFactorSteps"))


def test_what_the_model_takes_from_the_source():
    assert (SLOTS, MORE_SLOTS, RAWS, FACTORS) == (6, 8, 8, 8)
    assert "const Items items{n_steps, same_rows ? 4 : 2};" in SOURCE  # steps whose keys come before the first values
    assert "int i = warp - kProducer;\n    for (; i < 2 * n_steps; i += 2)" in SOURCE
    assert "for (int i = warp >> 1; i < 2 * n_steps; i += kWideners / 2)" in SOURCE
    for name, count in (("full", "kWideners / 2"), ("empty", "kStreams"), ("raw_empty", "kWideners / 2"), ("factors_full", "1"),
                        ("added", "1"), ("finished", "1")):
        assert re.search(rf"mbar_init\(smem_u32\(sh\.{name} \+ \w\), {re.escape(count)}\)", SOURCE), name


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        assert self.left > 0, "an arrival too many"
        self.left -= 1
        if self.left == 0:
            self.left = self.count
            self.phase += 1

    def passed(self, parity):
        return self.phase & 1 != parity


def run(n, same, n0, seed, by_kind=False):
    """n steps; `same`: both streams have the same rows and every other step, else stream 0 has the first n0 steps and
    stream 1 all of them.  `by_kind`: one producer takes the keys and one the values."""
    rng = random.Random(seed)
    lead, slots = (4, MORE_SLOTS) if same else (2, SLOTS)
    key = lambda s: s if s < lead else 2 * s - lead + 1        # noqa: E731  items in the order of their use
    value = lambda s: lead + 2 * s if s <= n - lead else n + s  # noqa: E731
    item = {key(s): (False, s) for s in range(n)} | {value(s): (True, s) for s in range(n)}
    assert sorted(item) == list(range(2 * n))
    steps = [list(range(x, n, 2)) for x in (0, 1)] if same else [list(range(n0)), list(range(n))]
    bars = lambda count, k: [Barrier(count) for _ in range(k)]  # noqa: E731
    # the pair's two warps arrive together here, and so does a copy with its expected bytes
    raw_full, raw_empty, full, empty = bars(1, RAWS), bars(1, RAWS), bars(1, slots), bars(2, slots)
    factors_full, added, finished = bars(1, FACTORS), bars(1, 2), bars(1, 2)
    scored, weighed = [bars(1, 2), bars(1, 2)], [bars(1, 2), bars(1, 2)]
    landed, read, widened, factors = set(), set(), set(), [None] * FACTORS
    scores_done, weights, products, used = set(), set(), set(), [set(), set()]
    given = [0] * (2 * n)
    copies, issued = [], [[], []]  # in flight

    def producer(items):
        for i in items:
            while not raw_empty[i % RAWS].passed((i // RAWS & 1) ^ 1):
                yield
            assert i < RAWS or i - RAWS in read, "a raw slot is filled before it was read"
            copies.append(i)
            yield

    def land(i):
        landed.add(i)
        raw_full[i % RAWS].arrive()

    def pair(w):
        for i in range(w, 2 * n, 2):
            is_value, s = item[i]
            while not raw_full[i % RAWS].passed(i // RAWS & 1):
                yield
            assert i in landed, "codes are read before they are there"
            while not empty[i % slots].passed((i // slots & 1) ^ 1):
                yield
            assert i < slots or given[i - slots] == 2, "a slot is widened into while products read it"
            yield
            widened.add(i)
            full[i % slots].arrive()
            if not is_value:
                old = factors[s % FACTORS]
                assert old is None or all(old in used[x] or old not in steps[x] for x in (0, 1)), "factors are overwritten"
                factors[s % FACTORS] = s
                yield
                factors_full[s % FACTORS].arrive()
            yield
            read.add(i)
            raw_empty[i % RAWS].arrive()

    def there(i):
        while not full[i % slots].passed(i // slots & 1):
            yield
        assert i in widened and i + slots not in widened, "a product of what is not there"

    def give(i, times):
        given[i] += times
        for _ in range(times):
            empty[i % slots].arrive()

    def mma(x):
        mine = steps[x]
        m, times = len(mine), 2 if same else 1

        def scores(j):
            i = key(mine[j])
            yield from there(i)
            if j >= 2:
                while not added[x].passed(j & 1):
                    yield
                assert (x, j - 2) in products, "scores over weights that are still read"
            issued[x].append(lambda: (scores_done.add((x, j)), scored[x][j & 1].arrive(), give(i, times)))
            yield

        def values(j):
            i = value(mine[j])
            yield from there(i)
            while not weighed[x][j & 1].passed(j >> 1 & 1):
                yield
            assert (x, j) in weights, "a product of weights that are not there"
            issued[x].append(lambda: (products.add((x, j)), added[x].arrive(), j + 1 == m and finished[x].arrive(), give(i, times)))
            yield

        for j in range(min(2, m)):
            yield from scores(j)
        for j in range(m):
            yield from values(j)
            if j + 2 < m:
                yield from scores(j + 2)
        for s in range(m, n) if not same else ():
            for i in (key(s), value(s)):
                yield from there(i)
                give(i, 1)
                yield

    def softmax(x):
        for j, s in enumerate(steps[x]):
            while not factors_full[s % FACTORS].passed(s // FACTORS & 1):
                yield
            assert factors[s % FACTORS] == s, "factors of another step"
            while not scored[x][j & 1].passed(j >> 1 & 1):
                yield
            assert (x, j) in scores_done, "scores are read before they are there"
            yield
            if j > 0 and rng.random() < 0.5:  # the output is rescaled
                while not added[x].passed((j - 1) & 1):
                    yield
                assert (x, j - 1) in products, "an output that is still added to"
            assert factors[s % FACTORS] == s, "factors of another step"
            used[x].add(s)
            weights.add((x, j))
            weighed[x][j & 1].arrive()
            yield
        while steps[x] and not finished[x].passed(0):
            yield
        assert not steps[x] or (x, len(steps[x]) - 1) in products, "an output that is not finished"

    turns = [[key(s) for s in range(n)], [value(s) for s in range(n)]] if by_kind else [range(w, 2 * n, 2) for w in (0, 1)]
    agents = [producer(t) for t in turns] + [f(x) for f in (pair, mma, softmax) for x in (0, 1)]
    pace = [rng.choice((1, 1, 3, 10, 40)) for _ in agents] + [rng.choice((1, 5, 30)) for _ in range(3)]
    live = list(range(len(agents)))
    for _ in range(200000):
        if not live:
            return
        who = rng.choices(live + [len(agents) + k for k in range(3)], [pace[a] for a in live] + pace[-3:])[0]
        if who == len(agents) and copies:
            land(copies.pop(rng.randrange(len(copies))))
        elif who > len(agents) and issued[who - len(agents) - 1]:
            issued[who - len(agents) - 1].pop(0)()
        elif who < len(agents) and next(agents[who], agents) is agents:
            live.remove(who)
    raise AssertionError("a wait that nothing ends")


@pytest.mark.parametrize("n", list(range(1, 21)) + [40])
def test_rows_that_both_streams_have(n):
    for seed in range(12):
        run(n, True, 0, seed)


@pytest.mark.parametrize("n", list(range(1, 21)) + [40])
def test_two_tiles_of_rows(n):
    for seed in range(12):
        run(n, False, (0, 1, n - 1, n, n // 2, max(0, n - 3))[seed % 6], seed)


def test_producers_by_kind_are_found_out():
    """One producer for keys and one for values share raw slots: some schedules end in a wait that passes too early."""
    found = set()
    for seed in range(300):
        try:
            run(30, True, 0, seed, by_kind=True)
        except AssertionError as e:
            found.add(str(e).split("\n")[0])
    assert found
