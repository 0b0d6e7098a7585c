"""The rings of csrc/paged_tiles.cu as a model, searched through every order of events: no tile is loaded into a
slot that a group has not released.

K and V tile of each key block go to slots; a producer each for K and V waits for its slot's phase by one parity bit.
Two groups use the tiles. A block of their own gives K and V back by commits, which arrive in order but at
any later time; a block of the other group's only gives both back at once, as soon as they are there."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "transformer_linear_layer_gb300", "csrc", "paged_tiles.cu")


def slots_in_source():
    """{head width: (slots of K's ring, of V's)}, or {} when there are no two rings."""
    m = re.search(r"KS = D == 64 \? (\d+) : (\d+), VS = D == 64 \? (\d+) : (\d+)", open(SOURCE).read())
    return {64: (int(m[1]), int(m[3])), 128: (int(m[2]), int(m[4]))} if m else {}


def separate(k, v):
    """Slot and phase of tile j of kind 0 (K) or 1 (V): a ring each."""
    return k + v, lambda kind, j: (j % k, j // k) if kind == 0 else (k + j % v, j // v)


def shared(n):
    """One ring that K and V tiles fill in turn."""
    return n, lambda kind, j: ((2 * j + kind) % n, (2 * j + kind) // n)


def overwrites(rings, programs):
    """Whether some order of events loads a tile into a slot that is still in use. programs: for each group, True
    for a block of its own, False for one that it only gives back."""
    n, place = rings
    blocks = len(programs[0])
    # a state: next block of each producer; for each group the blocks done, the commits that have not arrived
    # (tiles, in order); tiles that each group has given back
    start = ((0, 0), (0, 0), ((), ()), (frozenset(), frozenset()))
    seen, todo = {start}, [start]

    def phases(back, slot):
        """Phases of a slot that are over: tiles there that both groups have given back, from the first on."""
        c = 0
        for k in range(2 * blocks):
            tiles = [(kind, j) for kind in (0, 1) for j in range(blocks) if place(kind, j) == (slot, k)]
            if not tiles or not all(tiles[0] in b for b in back):
                return c
            c += 1
        return c

    while todo:
        at, done, pending, back = todo.pop()
        after = []
        for kind in (0, 1):
            j = at[kind]
            if j < blocks:
                slot, k = place(kind, j)
                c = phases(back, slot)
                if c & 1 == k & 1:  # the parity that the producer waits for
                    if c < k:
                        return True
                    after.append((tuple(x + (i == kind) for i, x in enumerate(at)), done, pending, back))
        for g in (0, 1):
            j = done[g]
            new_done = tuple(x + (i == g) for i, x in enumerate(done))
            if j < blocks and at[0] > j and at[1] > j:
                if programs[g][j]:
                    queue = pending[g] + ((0, j), (1, j))
                    after.append((at, new_done, tuple(queue if i == g else p for i, p in enumerate(pending)), back))
                else:
                    gone = tuple(b | {(0, j), (1, j)} if i == g else b for i, b in enumerate(back))
                    after.append((at, new_done, pending, gone))
            if pending[g]:
                gone = tuple(b | {pending[g][0]} if i == g else b for i, b in enumerate(back))
                after.append((at, done, tuple(p[1:] if i == g else p for i, p in enumerate(pending)), gone))
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return False


PROGRAMS = {
    "both": ([True] * 9, [True] * 9),
    "one ends first": ([True] * 9, [True] * 3 + [False] * 6),
    "in turn": ([True, False] * 4 + [True], [False, True] * 4 + [False]),
    "one is idle": ([True] * 9, [False] * 9),
}


@pytest.mark.parametrize("program", sorted(PROGRAMS))
@pytest.mark.parametrize("width", [64, 128])
def test_no_tile_is_overwritten(width, program):
    slots = slots_in_source()
    assert slots, "K and V tiles share slots"
    assert not overwrites(separate(*slots[width]), PROGRAMS[program])


def test_the_model_sees_a_slot_that_two_producers_share():
    assert overwrites(shared(5), PROGRAMS["one ends first"])
    assert not overwrites(shared(5), PROGRAMS["both"])
    assert not overwrites(shared(4), PROGRAMS["one ends first"])


def test_the_joining_kernel_reads_no_constants():
    """It may start before the attention kernel has written what it reads (it waits inside), so loads of data that is
    constant while a kernel runs are not for it."""
    join = open(os.path.join(os.path.dirname(SOURCE), "paged_join.cu")).read()
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", join)
