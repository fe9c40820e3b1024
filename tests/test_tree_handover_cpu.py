"""The hand-over of decoded steps in csrc/kv_tree_wide.cu, played on the CPU over the stretches that a CTA's run crosses.

A run is a list of stretches (one sequence, kv head and tile each), of one step or of hundreds.  The decoder warps walk them
without waiting for one another; what holds a warp back is the barrier of the place that it is about to write, of which it
sees the parity alone.  The numbering that is played is read from the kernel's source.
"""
import os
import random
import re

import pytest

import rotated_codebook_quantized_gb300 as tq

SRC = open(os.path.join(os.path.dirname(tq.__file__), "csrc", "kv_tree_wide.cu")).read()
CONST = {n: int(re.search(rf"constexpr int {n} = (\d+);", SRC).group(1)) for n in ("kTok", "kUnit", "kStages", "kDec")}
PER_STEP = CONST["kTok"] // CONST["kUnit"]


def _kernels_numbering():
    """first(d, g): warp d's first unit in a stretch that begins at the CTA's step g, as the decoders' loop has it."""
    start = re.search(r"for \(int u = u0 \+ (\w+); u < s1 \* kUnits; u \+= D\)", SRC).group(1)
    assert re.search(rf"int ahead = u0 \+ {start}[,;]", SRC), "the copies start where the decoding does"
    assert re.search(rf"stage = \(g \+ {start} / kUnits\) % kStages, phase = \(g \+ {start} / kUnits\) / kStages & 1", SRC)
    if start == "d":
        return lambda d, g: d
    expr = re.search(rf"const int {start} = (.+?);", SRC).group(1).replace("(int)", "").replace("/", "//")
    return lambda d, g: eval(expr, {}, dict(d=d, g=g, D=CONST["kDec"], kUnits=PER_STEP, **CONST))  # noqa: S307


class Broken(AssertionError):
    pass


def _play(stretches, shared, first, seed):
    """One order of the roles.  shared: both streams read every step (two tiles); otherwise each takes every other step of a
    stretch, and a stretch begins when both are done with the one before (its queries are written then)."""
    rnd = random.Random(seed)
    places, warps = CONST["kStages"], CONST["kDec"]
    bounds = [0]
    for s in stretches:
        bounds.append(bounds[-1] + s)
    # the units of each warp, the steps of each stream, in their order: (global step), (global step, stretch)
    todo = []
    for d in range(warps):
        mine = []
        for z, s in enumerate(stretches):
            mine += [bounds[z] + u // PER_STEP for u in range(first(d, bounds[z]), s * PER_STEP, warps)]
        todo.append(mine[::-1])
    reads = [[(i, z) for z in range(len(stretches)) for i in range(bounds[z] + (0 if shared else t), bounds[z + 1], 1 if shared else 2)][::-1]
             for t in range(2)]
    left = list(stretches) if not shared else [2 * s for s in stretches]  # reads of each stretch still to come
    written, whole, frees, freed = [0] * places, [0] * places, [0] * places, [0] * places
    seen = [[], []]  # steps whose keys a stream has begun to read and whose places it has not given back
    slow = [rnd.random() < 0.3 for _ in range(warps)]
    while any(todo) or any(reads) or any(seen):
        moves = []
        for d in range(warps):
            if todo[d]:
                k, p = divmod(todo[d][-1], places)
                if freed[p] % 2 != (k - 1) % 2:  # the barrier's phase of parity (k - 1) % 2 has completed
                    moves.append(("write", d))
        for t in range(2):
            if seen[t]:
                moves.append(("free", t))
            if reads[t]:
                i, z = reads[t][-1]
                k, p = divmod(i, places)
                # the next step's scores may be issued before the present step's values, in one stretch
                ahead = not seen[t] or len(seen[t]) == 1 and seen[t][0][1] == z
                if ahead and (shared or z == 0 or left[z - 1] == 0) and whole[p] % 2 != k % 2:
                    moves.append(("read", t))
        if not moves:
            raise Broken("every role waits")
        kind, who = rnd.choice(moves)
        if len(moves) > 1 and rnd.random() < 0.9 and (kind == "write" and slow[who] or kind != "write" and who == seed % 2):
            continue  # some roles are slow
        if kind == "write":
            k, p = divmod(todo[who].pop(), places)
            if freed[p] != k:
                raise Broken("a place was written before it was free")
            written[p] += 1
            if written[p] == PER_STEP:
                written[p], whole[p] = 0, whole[p] + 1
        elif kind == "read":
            i, z = reads[who].pop()
            k, p = divmod(i, places)
            if whole[p] != k + 1:
                raise Broken("a step was read before it was whole, or after it was written over")
            seen[who].append((i, z))
        else:
            i, z = seen[who].pop(0)
            k, p = divmod(i, places)
            if whole[p] != k + 1:
                raise Broken("a step was written over while it was in use")
            left[z] -= 1
            frees[p] += 1
            if frees[p] == (2 if shared else 1):
                frees[p], freed[p] = 0, freed[p] + 1


RUNS = [[1] * 16 + [44], [2] * 8 + [121], [2] * 6 + [8], [1] * 14 + [3], [5] * 8, [8] * 6, [7, 1, 1, 2, 40], [3, 4, 5] * 4, [40],
        [13, 1, 13, 2, 13], [1] * 60, [2] * 30]


@pytest.mark.parametrize("shared", [False, True], ids=["even_and_odd_steps", "two_tiles"])
@pytest.mark.parametrize("stretches", RUNS, ids=lambda s: "_".join(map(str, s))[:24])
def test_places_are_never_taken_early_across_stretches(stretches, shared):
    first = _kernels_numbering()
    for g in range(0, 40):  # every unit of a stretch belongs to one warp
        assert sorted(u for d in range(CONST["kDec"]) for u in range(first(d, g), 12 * PER_STEP, CONST["kDec"])) == list(range(12 * PER_STEP))
    for seed in range(20):
        _play(stretches, shared, first, seed)


@pytest.mark.parametrize("shared", [False, True], ids=["even_and_odd_steps", "two_tiles"])
def test_places_across_random_stretches(shared):
    first = _kernels_numbering()
    for seed in range(150):
        rnd = random.Random(1000 + seed)
        _play([rnd.choice([1, 1, 2, 2, 3, 5, 8, 13, 30]) for _ in range(rnd.randint(1, 24))], shared, first, seed)


def test_the_play_tells_a_numbering_that_starts_anew():
    """Units counted from each stretch's beginning leave rounds of a place out: the play has to see it."""
    for stretches in ([2] * 8 + [40], [1] * 16 + [44]):
        for shared in (False, True):
            with pytest.raises(Broken):
                for seed in range(20):
                    _play(stretches, shared, lambda d, g: d, seed)
