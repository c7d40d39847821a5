"""Host models of waits in the chunk kernel's tree kinds. Barriers behave as mbarriers do (a phase ends with its count's arrival, a
waiter sees the phase's parity), roles run in random order at random speeds.

Trees of two query tiles over an FP8 cache: the softmax threads of tiles A and B write their tile's query terms and arrive, the MMA
warp waits and multiplies; tile B's threads pass items in which B has no queries without waiting for anything but the ring that
hands items on. Every multiplication has to find its own item's terms in place, and no term may be overwritten that is still to be
read. Trees of one query tile: an item's O may be read only when its last P V is done."""
import random

import pytest

SLOTS, THREADS = 4, 3  # of the ring that hands items on; threads of a tile in the model


class Barrier:
    def __init__(self, count):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1

    def passed(self, parity):
        """What a wait on `parity` sees: true once the phase of that parity is no longer the current one."""
        return (self.phase & 1) != (parity & 1)


class Fault(Exception):
    pass


def run(has_b, tiles, one_barrier, seed):
    """One CTA over the items: has_b[i] whether tile B has queries in item i, tiles[i] its K/V tiles. one_barrier: both tiles'
    threads arrive on one barrier, in every item; else a barrier a tile, and only tiles with queries take part."""
    rng = random.Random(seed)
    n = len(has_b)
    taken = [0] * (2 * THREADS + 1)         # items each role has taken from the ring
    ready = [Barrier(2 * THREADS)] if one_barrier else [Barrier(THREADS), Barrier(THREADS)]
    scores, done = [Barrier(1), Barrier(1)], [Barrier(1), Barrier(1)]
    weights = [Barrier(THREADS), Barrier(THREADS)]
    terms = [[-1] * THREADS for _ in range(2)]  # the item whose terms a thread has written

    def posted(i):
        return i < min(taken) + SLOTS

    def softmax(x, t):
        me, g = x * THREADS + t, 0
        for i in range(n):
            while not posted(i):
                yield
            taken[me] += 1
            yield
            takes_part = x == 0 or has_b[i]
            if takes_part or one_barrier:
                terms[x][t] = i
                yield
                ready[0 if one_barrier else x].arrive()
            if not takes_part:
                continue
            for _ in range(tiles[i]):
                while not scores[x].passed(g):
                    yield
                weights[x].arrive()
                g += 1
                yield
            while not done[x].passed(g - 1):
                yield

    def mma():
        g, units, b_units = [0, 0], 0, 0
        for i in range(n):
            while not posted(i):
                yield
            taken[-1] += 1
            yield
            while not ready[0].passed(units):
                yield
            units += 1
            if has_b[i] and not one_barrier:
                while not ready[1].passed(b_units):
                    yield
                b_units += 1
            xs = [0, 1] if has_b[i] else [0]
            for x in xs:
                if terms[x] != [i] * THREADS:
                    raise Fault(f"item {i}: tile {'AB'[x]} is multiplied with the terms of items {terms[x]}")
                scores[x].arrive()
                yield
            for j in range(tiles[i]):
                for x in xs:
                    while not weights[x].passed(g[x]):
                        yield
                    if terms[x] != [i] * THREADS:
                        raise Fault(f"item {i}: terms of tile {'AB'[x]} were overwritten")
                    g[x] += 1
                    done[x].arrive()
                    if j + 1 < tiles[i]:
                        scores[x].arrive()
                    yield

    roles = [softmax(x, t) for x in range(2) for t in range(THREADS)] + [mma()]
    speed = [rng.random() ** 2 + 0.01 for _ in roles]
    live, idle = set(range(len(roles))), 0
    while live:
        k = rng.choices(sorted(live), [speed[r] for r in sorted(live)])[0]
        before = (tuple(taken), tuple(b.phase for b in scores + done), tuple(map(tuple, terms)))
        try:
            next(roles[k])
        except StopIteration:
            live.discard(k)
        after = (tuple(taken), tuple(b.phase for b in scores + done), tuple(map(tuple, terms)))
        idle = idle + 1 if after == before else 0
        if idle > 20000:
            raise Fault("nobody moves")


def patterns(rng, kind, n=10):
    """Whether tile B has queries, item after item, and the items' K/V tiles."""
    b = {"none": [False] * n, "all": [True] * n, "mixed": [rng.random() < 0.5 for _ in range(n)]}[kind]
    return b, [rng.randint(1, 3) for _ in range(n)]


@pytest.mark.parametrize("kind", ["none", "all", "mixed"])
def test_a_barrier_for_each_tile(kind):
    for seed in range(50):
        run(*patterns(random.Random(seed), kind), one_barrier=False, seed=seed)


def test_one_barrier_for_both_tiles_would_not_do():
    """Tile B's arrivals for later items end the phase that stands for tile A's terms."""
    faults = 0
    for seed in range(50):
        try:
            run(*patterns(random.Random(seed), "none"), one_barrier=True, seed=seed)
        except Fault:
            faults += 1
    assert faults > 0


def test_the_model_with_queries_in_both_tiles():
    """Where both tiles always have queries one barrier would have been enough: both wait for the item's scores."""
    for seed in range(30):
        run(*patterns(random.Random(seed), "all"), one_barrier=True, seed=seed)


def run_one_tile(tiles, alternate, seed):
    """Trees of one query tile: scores run two K/V tiles ahead, so that a thread may have handed on its last weights while the P V of
    the tile before is still waiting for slower threads. An item's O is read behind a wait for its last P V. alternate: even and odd
    tiles' P V complete on a barrier each; else all on one."""
    rng = random.Random(seed)
    scores, weights = [Barrier(1), Barrier(1)], [Barrier(THREADS), Barrier(THREADS)]
    done = [Barrier(1), Barrier(1)]
    finished = [0]       # P V complete, in order
    issued = []          # P V on their way
    total = sum(tiles)

    def softmax(_):
        g = 0
        for n in tiles:
            for _ in range(n):
                while not scores[g & 1].passed(g >> 1):
                    yield
                weights[g & 1].arrive()
                g += 1
                yield
            last = g - 1
            bar, parity = (done[last & 1], last >> 1) if alternate else (done[0], last)
            while not bar.passed(parity):
                yield
            if finished[0] < g:
                raise Fault(f"O is read before the P V of tile {last}: {finished[0]} are done")

    def mma():
        g = 0  # K/V tiles whose P V is issued
        for n in tiles:
            for _ in range(min(2, n)):
                scores[(g + _) & 1].arrive()
                yield
            for j in range(n):
                while not weights[g & 1].passed(g >> 1):
                    yield
                issued.append(g)
                yield
                if j + 2 < n:
                    while finished[0] <= g:  # scores complete behind the P V issued before them
                        yield
                    scores[g & 1].arrive()
                g += 1

    def tensor_core():
        while finished[0] < total:
            if issued:
                g = issued.pop(0)
                finished[0] += 1
                done[g & 1 if alternate else 0].arrive()
            yield

    roles = [softmax(t) for t in range(THREADS)] + [mma(), tensor_core()]
    speed = [rng.random() ** 2 + 0.01 for _ in roles]
    live, left = set(range(len(roles))), 200000
    while live:
        left -= 1
        if left == 0:
            raise Fault("nobody moves")
        k = rng.choices(sorted(live), [speed[r] for r in sorted(live)])[0]
        try:
            next(roles[k])
        except StopIteration:
            live.discard(k)


def test_the_last_p_v_is_waited_for():
    for seed in range(150):
        rng = random.Random(seed)
        run_one_tile([rng.randint(1, 4) for _ in range(6)], True, seed)


def test_one_barrier_for_all_p_v_would_not_do():
    """Its parity takes the P V two tiles back for the last one's."""
    faults = 0
    for seed in range(150):
        rng = random.Random(seed)
        try:
            run_one_tile([rng.randint(2, 4) for _ in range(6)], False, seed)
        except Fault:
            faults += 1
    assert faults > 0
