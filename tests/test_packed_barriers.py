"""The barrier protocol of k_packed_attn.cu as a model, under random schedules (CPU): see
test_paged_barriers.py, whose barriers and schedules these are.  The roles follow the kernel wait by
wait; a change to its barriers belongs here first."""
import random

import pytest

from test_paged_barriers import SEEDS, Bar, Ring, Schedule, bars  # noqa: F401


class Arrival:
    """An asynchronous copy that arrives, when it lands, as a thread does."""

    def __init__(self, bar):
        self.bar = bar

    def land(self):
        self.bar.arrive()


SLOTS = 32     # tiles that are planned, and those whose scales are held


def packed(seed, units, stages, most, buffers=4, late=False):
    """Units of so many key tiles, in steps of up to `most`.  `late`: the softmax reuses the weights' buffer as
    soon as its product is done, before the epilogue has taken the step's sums."""
    s, ring = Schedule(seed), Ring(16)
    ks, vs = stages
    kfull, kempty, vfull, vempty = bars(ks, 17), bars(ks, 1), bars(8, most), bars(vs, 1)
    sfull, sempty = bars(buffers, 2), bars(buffers, 4)
    qfull, qempty = bars(2, 2), bars(2, 8)
    pfull, ofull, oempty = bars(2, 4), bars(2, 1), bars(2, 4)
    tfull, tempty, tile = bars(SLOTS, 1), bars(SLOTS, 2), {}
    meet, held = bars(2, 4), {}

    edges = {}                                  # steps in which rows of V are cleared

    def steps(count):
        return [min(most, count - t) for t in range(0, count, most)]

    def planner():                              # the units, and a ring of their tiles
        n = 0
        for k, count in enumerate(units):
            yield from ring.put(k)
            for t in range(count):
                if n >= SLOTS:
                    yield tempty[n % SLOTS], n // SLOTS - 1
                last = t % most == most - 1 or t + 1 == count
                tile[n % SLOTS] = most - 1 - t % most if last else -1      # what its step lacks
                tfull[n % SLOTS].arrive()
                n += 1
        yield from ring.put(len(units))
        for _ in range(2):                      # the end, for either tile of a pair
            if n >= SLOTS:
                yield tempty[n % SLOTS], n // SLOTS - 1
            tile[n % SLOTS] = None
            tfull[n % SLOTS].arrive()
            n += 1

    def loads(kind, empty):                     # two tiles at a time
        n, size, step = 0, len(empty), 0
        while True:
            pair = []
            for m in (n, n + 1):
                yield tfull[m % SLOTS], m // SLOTS
                if tile[m % SLOTS] is not None:
                    pair.append((m, tile[m % SLOTS]))
            for m, _ in pair:
                if m >= size:
                    yield empty[m % size], m // size - 1
            for m, lack in pair:
                if kind == "k":
                    # the scales of the tile that had this place are no longer looked at
                    assert held.get(m % SLOTS, 0) == 0, "scales overwritten"
                    held[m % SLOTS] = 4
                    s.copies += [Arrival(kfull[m % size]) for _ in range(16)]
                    s.load(kfull[m % size])
                else:
                    s.load(vfull[step % 8])
                    for _ in range(lack):
                        vfull[step % 8].arrive()
                step += lack >= 0
                tempty[m % SLOTS].arrive()
            n += len(pair)
            if len(pair) < 2:
                return

    def scores():
        n = step = nq = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            if not count:
                continue
            yield qfull[nq & 1], nq >> 1
            for kt in steps(count):
                if step >= buffers:
                    yield sempty[step % buffers], step // buffers - 1
                for _ in range(kt):
                    yield kfull[n % ks], n // ks
                    s.commits.append(kempty[n % ks])
                    n += 1
                sfull[step % buffers].arrive()
                s.commits.append(sfull[step % buffers])
                step += 1
            nq += 1
        yield from ring.get(len(units))

    def values():
        step = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            for kt in steps(count):
                yield vfull[step % 8], step // 8
                yield pfull[step & 1], step >> 1
                s.commits.append(ofull[step & 1])
                step += 1
        yield from ring.get(len(units))

    def queries():
        nq = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            if not count:
                continue
            if nq >= 2:
                yield qempty[nq & 1], (nq >> 1) - 1
            yield from s.work(6)
            qfull[nq & 1].arrive()
            nq += 1
        yield from ring.get(len(units))

    def softmax(g):
        n = step = nq = met = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            if not count:
                continue
            yield qfull[nq & 1], nq >> 1
            for kt in steps(count):
                n += kt
                if (step & 1) == g:
                    mine = range(n - kt, n)
                    yield sfull[step % buffers], step // buffers
                    yield from s.work(5)
                    meet[g].arrive()
                    yield meet[g], met
                    met += 1
                    if step >= 2:
                        yield (ofull if late else oempty)[g], (step >> 1) - 1
                    if edges[step] if step in edges else edges.setdefault(step, s.rng.random() < 0.3):
                        yield vfull[step % 8], step // 8
                    yield from s.work(5)
                    for m in mine:
                        held[m % SLOTS] -= 1
                    pfull[g].arrive()
                    sempty[step % buffers].arrive()
                step += 1
            qempty[nq & 1].arrive()
            nq += 1
        yield from ring.get(len(units))

    def epilogue(w):
        n = step = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            for kt in steps(count):
                yield pfull[step & 1], step >> 1
                yield ofull[step & 1], step >> 1
                yield from s.work(8)
                oempty[step & 1].arrive()
                for m in range(n, n + kt if w == 0 else n):
                    vempty[m % vs].arrive()
                n += kt
                step += 1
            yield from s.work(10)
        yield from ring.get(len(units))

    s.run([planner(), loads("k", kempty), loads("v", vempty), scores(), values()] +
          [softmax(w // 4) for w in range(8)] + [epilogue(w) for w in range(4)] +
          [queries() for _ in range(2)])


@pytest.mark.parametrize("most,buffers", [(1, 2), (1, 4), (2, 4), (4, 4)])
@pytest.mark.parametrize("stages", [(4, 5), (4, 7), (8, 8)])
@pytest.mark.parametrize("seed", SEEDS)
def test_packed_attention(seed, stages, most, buffers):
    r = random.Random(seed)
    packed(seed, [r.choice([0, 1, 1, 2, 3, 4, 8]) for _ in range(30)], stages, most, buffers)
    packed(seed, [r.choice([0, 1, 1, 2]) for _ in range(60)], stages, most, buffers)
    packed(seed, [1] * 40, stages, most, buffers)
    packed(seed, [37, 64], stages, most, buffers)


def test_a_buffer_that_is_used_again_too_early_mistakes_a_phase():
    with pytest.raises(AssertionError, match="phase|deadlock"):
        for seed in range(200):
            packed(seed, [9, 1, 1, 30, 2], (4, 7), 1, late=True)
