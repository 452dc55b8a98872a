"""The ring of keys and values of the tcgen05 attention kernel, as a model: copies that land in any order, warps that go on as soon as what they
wait for answers, and barriers that answer by a phase's parity, as the hardware's do - a wait a turn early is answered "complete".

No product may read a slot that does not hold its tile.  With a barrier for each slot the model finds one that does, for a ring of an odd
number of slots and an item of one tile of rows; with the kernel's barriers, one for each of two turns of the ring, it finds none."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bf16_weight_exponent_gb300", "csrc")


class Barrier:
    def __init__(self):
        self.done = 0                       # phases completed

    def answers(self, phase):
        return (self.done & 1) != (phase & 1)


def run(NS, tiles, N, per_turns, seed):
    """One schedule; the tiles (kind, n) that a product read before they were there."""
    rng = random.Random(seed)
    barriers = per_turns * NS
    full, of, turn = [Barrier() for _ in range(barriers)], lambda i: i % barriers, lambda i: i // barriers
    holds, consumed, wrong = {}, set(), []
    landed = {}
    s_read, p_there, pv_done, s_there = [0] * tiles, [0] * tiles, [0] * tiles, [0] * tiles
    reads = [0]                             # scores read by the softmax warps, of both tiles
    flying = []

    def copies():
        for i in range(2 * N):
            yield lambda i=i: i < NS or i - NS in consumed
            flying.append(i)

    def lands():
        while len(landed) < 2 * N:
            yield lambda: bool(flying)
            # values may be long in coming: they are put right before they count
            i = rng.choice([x for x in flying if x % 2 == 0] or flying) if rng.random() < 0.8 else rng.choice(flying)
            flying.remove(i)
            landed[i] = True
            holds[i % NS] = i
            full[of(i)].done += 1

    def read(i):
        if holds.get(i % NS) != i:
            wrong.append(i)

    def scores():
        q = 0
        for n in range(N):
            for t in range(tiles):
                yield lambda n=n: full[of(2 * n)].answers(turn(2 * n))
                yield lambda q=q: reads[0] >= q
                read(2 * n)
                s_there[t] += 1
                q += 1
            consumed.add(2 * n)

    def values():
        for n in range(N):
            for t in range(tiles):
                yield lambda n=n: full[of(2 * n + 1)].answers(turn(2 * n + 1))
                yield lambda t=t, n=n: p_there[t] > n
                read(2 * n + 1)
                pv_done[t] += 1
            consumed.add(2 * n + 1)

    def softmax(t):
        for n in range(N):
            yield lambda n=n: s_there[t] > n
            reads[0] += 1
            yield lambda n=n: pv_done[t] >= n
            p_there[t] += 1

    actors = [copies(), lands(), scores(), values()] + [softmax(t) for t in range(tiles)]
    waits = {a: next(a) for a in actors}
    while waits and not wrong:
        ready = [a for a, w in waits.items() if w()]
        assert ready, "nobody can go on"
        a = rng.choice(ready)
        try:
            waits[a] = next(a)
        except StopIteration:
            del waits[a]
    return wrong


@pytest.mark.parametrize("tiles", [1, 2])
@pytest.mark.parametrize("NS", [5, 6, 10, 11])
def test_no_tile_is_read_early(NS, tiles):
    for seed in range(400):
        assert run(NS, tiles, 14, 2, seed) == []


def test_the_model_finds_a_turn_early():
    assert any(run(5, 1, 14, 1, seed) for seed in range(400))
    assert not any(run(5, 2, 14, 1, seed) for seed in range(400))
    assert not any(run(6, 1, 14, 1, seed) for seed in range(400))


def test_the_kernel_has_these_barriers():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "k_attend_tc.cu")).read())
    uses = re.findall(r"(?<![qsp])\bfull\[([^]]*)\]", text)
    assert len(uses) >= 7
    assert all("% (2 * NS)" in u for u in uses if u not in ("i", "NS + i")) and uses.count("i") == uses.count("NS + i") == 1
    turns = re.findall(r"/ \(2 \* NS\)\) & 1", text)
    assert len(turns) == 3 and "empty = full + 2 * NS" in text
    assert not re.search(r"/ NS\) & 1[^)]*\)[^;]*full", text)
