"""The barrier protocols of the paged-cache kernels as a model, under random schedules (CPU).

An mbarrier knows its phase by one parity bit, so a role that tests for phase f is right only while
f is the phase under way or the one just completed.  The model's barriers count their phases and
check that at every test.  Each kernel's roles are generators that yield what they wait for, a
(barrier, phase) pair, or None for work of some length; copies land and the tensor core's commits
arrive in their own time.  A schedule that ends with a role still waiting is a deadlock.

The roles follow k_paged_attn.cu, k_paged_attn_tc.cu and k_paged_mass.cu wait by wait; a change to
their barriers belongs here first."""
import random

import pytest

UNITS = 8      # places of the ring that hands units to the roles


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.tx, self.done = count, count, 0, 0

    def _complete(self):
        if self.pending == 0 and self.tx == 0:
            self.done, self.pending = self.done + 1, self.count

    def arrive(self):
        assert self.pending > 0, "more arrivals than the barrier counts"
        self.pending -= 1
        self._complete()

    def expect(self):
        self.tx += 1
        self.arrive()

    def land(self):
        self.tx -= 1
        self._complete()

    def passed(self, phase):
        by_parity = (self.done & 1) != (phase & 1)
        assert by_parity == (self.done > phase), "phase %d taken for %d" % (self.done, phase)
        assert self.done <= phase + 1, "phase %d passed unseen" % phase
        return by_parity


def bars(n, count):
    return [Bar(count) for _ in range(n)]


class Ring:
    def __init__(self, readers):
        self.full, self.empty = bars(UNITS, 1), bars(UNITS, readers)

    def put(self, k):
        if k >= UNITS:
            yield self.empty[k % UNITS], k // UNITS - 1
        self.full[k % UNITS].arrive()

    def get(self, k):
        yield self.full[k % UNITS], k // UNITS
        self.empty[k % UNITS].arrive()


class Schedule:
    """Random turns of the roles, of copies in flight and of the tensor core's commits (in order)."""

    def __init__(self, seed):
        self.rng, self.copies, self.commits = random.Random(seed), [], []

    def load(self, bar):
        bar.expect()
        self.copies.append(bar)

    def work(self, most):
        for _ in range(self.rng.randrange(most)):
            yield None

    def run(self, roles):
        roles = [[r, None] for r in roles]
        idle = 0
        while roles:
            turn = self.rng.randrange(len(roles) + 2)
            idle += 1
            assert idle < 20000 * (1 + len(roles)), "deadlock"
            if turn == len(roles):
                if self.copies:
                    self.copies.pop(self.rng.randrange(len(self.copies))).land()
                    idle = 0
            elif turn == len(roles) + 1:
                if self.commits:
                    self.commits.pop(0).arrive()
                    idle = 0
            else:
                role = roles[turn]
                if role[1] is None or role[1][0].passed(role[1][1]):
                    idle = 0
                    try:
                        role[1] = next(role[0])
                    except StopIteration:
                        roles.pop(turn)


def short_chunks(seed, units, k_stages, v_stages, skip=False):
    """k_paged_attn: units of (key tiles, joins of rows at the end).  `skip`: a warp does not look at
    the other team's tiles, which took an unfinished phase for a finished one."""
    s, ring, meet = Schedule(seed), Ring(9), Bar(8)
    kfull, kempty = bars(k_stages, 1), bars(k_stages, 4 if skip else 8)
    vfull, vempty = bars(v_stages, 1), bars(v_stages, 4 if skip else 8)
    qfull, qempty = bars(2, 1), bars(2, 8)

    def keys():
        nq = n = 0
        for k, (tiles, _) in enumerate(units):
            yield from ring.put(k)
            if tiles:
                if nq >= 2:
                    yield qempty[nq % 2], nq // 2 - 1
                s.load(qfull[nq % 2])
                nq += 1
            for _ in range(tiles):
                if n >= k_stages:
                    yield kempty[n % k_stages], n // k_stages - 1
                s.load(kfull[n % k_stages])
                n += 1
        yield from ring.put(len(units))

    def values():
        n = 0
        for k, (tiles, _) in enumerate(units):
            yield from ring.get(k)
            for _ in range(tiles):
                if n >= v_stages:
                    yield vempty[n % v_stages], n // v_stages - 1
                s.load(vfull[n % v_stages])
                n += 1
        yield from ring.get(len(units))

    def warp(team):
        n = nq = met = 0
        for k, (tiles, joins) in enumerate(units):
            yield from ring.get(k)
            if tiles:
                yield qfull[nq % 2], nq // 2
            for t in range(tiles):
                mine = t % 2 == team
                if mine or not skip:
                    yield kfull[n % k_stages], n // k_stages
                    yield from s.work(8 if mine else 1)
                    kempty[n % k_stages].arrive()
                    yield vfull[n % v_stages], n // v_stages
                    yield from s.work(8 if mine else 1)
                    vempty[n % v_stages].arrive()
                n += 1
            if tiles:
                qempty[nq % 2].arrive()
                nq += 1
            for _ in range(1 + 2 * joins):
                meet.arrive()
                yield meet, met
                met += 1
        yield from ring.get(len(units))

    s.run([keys(), values()] + [warp(w // 4) for w in range(8)])


def long_chunks(seed, units, slots):
    """k_paged_attn_tc: units of (key tiles, row tiles, which key tiles some row does not see)."""
    s, ring = Schedule(seed), Ring(9)
    full, empty, qfull, qempty = bars(slots, 1), bars(slots, 1), Bar(1), Bar(1)
    sfull, pfull, ofull = bars(2, 1), bars(2, 4), bars(2, 1)
    clean = [bars(2, 4), bars(2, 4)]

    def producer():
        nq = n = 0
        for k, (tiles, _, _) in enumerate(units):
            yield from ring.put(k)
            if tiles:
                if nq:
                    yield qempty, nq - 1
                s.load(qfull)
                nq += 1
            for _ in range(2 * tiles):          # K and V in turn
                if n >= slots:
                    yield empty[n % slots], n // slots - 1
                s.load(full[n % slots])
                n += 1
        yield from ring.put(len(units))

    def issuer():
        nq = n = 0
        seen = [0, 0]
        for k, (tiles, rows, _) in enumerate(units):
            yield from ring.get(k)
            if not tiles:
                continue
            yield qfull, nq
            nq += 1
            yield full[n % slots], n // slots
            s.commits += sfull[:rows] + [empty[n % slots]] + ([qempty] if tiles == 1 else [])
            n += 1
            for j in range(tiles):
                more = j + 1 < tiles
                for t in range(rows):
                    yield pfull[t], seen[t]
                    seen[t] += 1
                    if more and t == 0:
                        yield full[(n + 1) % slots], (n + 1) // slots
                    s.commits.append(sfull[t] if more else ofull[t])
                s.commits.append(empty[n % slots])
                if more:
                    s.commits.append(empty[(n + 1) % slots])
                    if j + 2 == tiles:
                        s.commits.append(qempty)
                n += 2 if more else 1
        yield from ring.get(len(units))

    def softmax(t):
        ns = no = n = edges = 0
        for k, (tiles, rows, edge) in enumerate(units):
            yield from ring.get(k)
            if t < rows:
                for j in range(tiles):
                    yield sfull[t], ns
                    ns += 1
                    v = n + 2 * j + 1
                    yield full[v % slots], v // slots
                    if edge[j] and rows == 2:
                        yield from s.work(6)
                        clean[t][edges & 1].arrive()
                        yield clean[t ^ 1][edges & 1], edges >> 1
                        edges += 1
                    yield from s.work(10)
                    pfull[t].arrive()
                if tiles:
                    yield ofull[t], no
                    no += 1
                yield from s.work(20)
            n += 2 * tiles
        yield from ring.get(len(units))

    s.run([producer(), issuer()] + [softmax(w // 4) for w in range(8)])


def mass(seed, units, stages):
    """k_paged_mass: units of (steps of rows, key tiles)."""
    s, ring, ahead = Schedule(seed), Ring(11), 8
    kfull, kempty, qfull, qempty = bars(stages, 1), bars(stages, 1), bars(2, 1), bars(2, 1)
    sfull, sfree = bars(4, 1), bars(4, 4)
    lfull, lempty, ufull, uempty = bars(ahead, 1), bars(ahead, 8), bars(ahead, 1), bars(ahead, 8)

    def producer():
        n = 0
        for k, (steps, tiles) in enumerate(units):
            yield from ring.put(k)
            for _ in range(tiles if steps else 0):
                if n >= stages:
                    yield kempty[n % stages], n // stages - 1
                s.load(kfull[n % stages])
                n += 1
        yield from ring.put(len(units))

    def issuer():
        n = nq = n2 = 0
        for k, (steps, tiles) in enumerate(units):
            yield from ring.get(k)
            if not steps:
                continue
            for i in range(tiles):
                yield kfull[(n + i) % stages], (n + i) // stages
            for _ in range(steps):
                b0, b1 = (nq & 1) * 2, (n2 & 1) * 2 + 1
                yield qfull[nq % 2], nq // 2
                if nq >= 2:
                    yield sfree[b0], (nq >> 1) - 1
                s.commits.append(sfull[b0])
                if tiles == 2:
                    if n2 >= 2:
                        yield sfree[b1], (n2 >> 1) - 1
                    s.commits.append(sfull[b1])
                    n2 += 1
                s.commits.append(qempty[nq % 2])
                nq += 1
            s.commits += [kempty[(n + i) % stages] for i in range(tiles)]
            n += tiles
        yield from ring.get(len(units))

    def old_weights():                          # a unit's are handed on when the next one is known
        for k in range(len(units) + 1):
            yield from ring.get(k)
            if k:
                if k - 1 >= ahead:
                    yield uempty[(k - 1) % ahead], (k - 1) // ahead - 1
                ufull[(k - 1) % ahead].arrive()

    def rows():
        n = 0

        def hand_on(k):
            if k >= ahead:
                yield lempty[k % ahead], k // ahead - 1
            lfull[k % ahead].arrive()
        for k, (steps, _) in enumerate(units):
            yield from ring.get(k)
            for i in range(steps):
                if n >= 2:
                    yield qempty[n % 2], n // 2 - 1
                s.load(qfull[n % 2])
                if i:
                    yield from hand_on(n - 1)
                n += 1
            if steps:
                yield from hand_on(n - 1)
        yield from ring.get(len(units))

    def sums(g):
        n = ns = 0
        for k, (steps, tiles) in enumerate(units):
            yield from ring.get(k)
            for _ in range(steps):
                yield lfull[n % ahead], n // ahead
                if g < tiles:
                    buf = (ns & 1) * 2 + g
                    yield sfull[buf], ns >> 1
                    yield from s.work(8)
                    sfree[buf].arrive()
                    ns += 1
                lempty[n % ahead].arrive()
                n += 1
            yield ufull[k % ahead], k // ahead
            uempty[k % ahead].arrive()
        yield from ring.get(len(units))

    s.run([producer(), issuer(), old_weights(), rows()] + [sums(w // 4) for w in range(8)])


SEEDS = range(12)


@pytest.mark.parametrize("stages", [(3, 3), (3, 2), (6, 5)])
@pytest.mark.parametrize("seed", SEEDS)
def test_short_chunks(seed, stages):
    r = random.Random(seed)
    short_chunks(seed, [(r.choice([0, 1, 2, 3, 6, 8]), r.choice([1, 1, 2, 4])) for _ in range(25)],
                 *stages)
    short_chunks(seed, [(r.choice([0, 1, 1, 2]), 1) for _ in range(40)], *stages)


def test_a_team_that_passes_over_stages_mistakes_a_phase():
    with pytest.raises(AssertionError, match="phase"):
        for seed in range(200):
            short_chunks(seed, [(40, 1), (7, 1), (40, 1)], 3, 3, skip=True)


@pytest.mark.parametrize("slots", [4, 8])
@pytest.mark.parametrize("seed", SEEDS)
def test_long_chunks(seed, slots):
    r = random.Random(seed)
    units = []
    for _ in range(25):
        tiles = r.choice([0, 1, 1, 2, 3, 7])
        units.append((tiles, r.choice([1, 2]), [r.random() < 0.4 for _ in range(tiles)]))
    long_chunks(seed, units, slots)


@pytest.mark.parametrize("stages", [2, 3, 4, 8])
@pytest.mark.parametrize("seed", SEEDS)
def test_mass(seed, stages):
    r = random.Random(seed)
    mass(seed, [(r.choice([0, 1, 1, 1, 2, 3, 5]), r.choice([1, 2, 2])) for _ in range(40)], stages)
    mass(seed, [(r.choice([0, 0, 0, 1, 2]), r.choice([1, 2])) for _ in range(50)], stages)
