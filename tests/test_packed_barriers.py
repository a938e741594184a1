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


SLOTS = 16     # tiles whose scales are held


def packed(seed, units, stages, most, late=False):
    """Units of so many key tiles, in steps of up to `most`.  `late`: the softmax reuses the weights' buffer as
    soon as its product is done, before the epilogue has taken the step's sums."""
    s, ring = Schedule(seed), Ring(19)
    ks, vs = stages
    kfull, kempty, vfull, vempty = bars(ks, 9), bars(ks, 1), bars(vs, 9), bars(vs, 1)
    qfull, qempty = bars(2, 4), bars(2, 8)
    sfull, pfull, ofull, oempty = bars(2, 2), bars(2, 4), bars(2, 1), bars(2, 4)
    meet, held = bars(2, 4), {"k": {}, "v": {}}

    def steps(count):
        return [min(most, count - t) for t in range(0, count, most)]

    def tiles(name, full, empty, unit):
        n, size, k = 0, len(full), 0

        def fetch():                            # the next unit with tiles; the one after the last is the end
            nonlocal k
            while True:
                yield from unit(k)
                k += 1
                if k > len(units) or units[k - 1]:
                    return

        yield from fetch()
        while k <= len(units):
            count = units[k - 1]
            for t in range(count):
                if t + 1 == count:
                    yield from fetch()
                if n >= size:
                    yield empty[n % size], n // size - 1
                # the scales of the tile that had this place are no longer looked at
                assert held[name].get(n % SLOTS, 0) == 0, "scales overwritten"
                held[name][n % SLOTS] = 4
                s.load(full[n % size])
                s.copies += [Arrival(full[n % size]) for _ in range(8)]
                n += 1

    def scores():
        n = step = nq = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            if not count:
                continue
            yield qfull[nq & 1], nq >> 1
            for kt in steps(count):
                if step >= 2:
                    yield pfull[step & 1], (step >> 1) - 1
                for _ in range(kt):
                    yield kfull[n % ks], n // ks
                    s.commits.append(kempty[n % ks])
                    n += 1
                sfull[step & 1].arrive()
                s.commits.append(sfull[step & 1])
                step += 1
            nq += 1
        yield from ring.get(len(units))

    def values():
        n = step = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            for kt in steps(count):
                yield pfull[step & 1], step >> 1
                for _ in range(kt):
                    yield vfull[n % vs], n // vs
                    s.commits.append(vempty[n % vs])
                    n += 1
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
                    yield sfull[g], step >> 1
                    yield from s.work(5)
                    for m in mine:
                        held["k"][m % SLOTS] -= 1
                        yield vfull[m % vs], m // vs
                    meet[g].arrive()
                    yield meet[g], met
                    met += 1
                    if step >= 2:
                        yield (ofull if late else oempty)[g], (step >> 1) - 1
                    yield from s.work(5)
                    for m in mine:
                        held["v"][m % SLOTS] -= 1
                    pfull[g].arrive()
                step += 1
            qempty[nq & 1].arrive()
            nq += 1
        yield from ring.get(len(units))

    def epilogue():
        step = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            for _ in steps(count):
                yield pfull[step & 1], step >> 1
                yield ofull[step & 1], step >> 1
                yield from s.work(8)
                oempty[step & 1].arrive()
                step += 1
            yield from s.work(10)
        yield from ring.get(len(units))

    s.run([tiles("k", kfull, kempty, ring.put), tiles("v", vfull, vempty, ring.get), scores(), values()] +
          [softmax(w // 4) for w in range(8)] + [epilogue() for _ in range(4)] +
          [queries() for _ in range(4)])


@pytest.mark.parametrize("most", [1, 2, 4])
@pytest.mark.parametrize("stages", [(4, 5), (8, 8)])
@pytest.mark.parametrize("seed", SEEDS)
def test_packed_attention(seed, stages, most):
    r = random.Random(seed)
    packed(seed, [r.choice([0, 1, 1, 2, 3, 4, 8]) for _ in range(30)], stages, most)
    packed(seed, [r.choice([0, 1, 1, 2]) for _ in range(60)], stages, most)
    packed(seed, [1] * 40, stages, most)
    packed(seed, [37, 64], stages, most)


def test_a_buffer_that_is_used_again_too_early_mistakes_a_phase():
    with pytest.raises(AssertionError, match="phase|deadlock"):
        for seed in range(200):
            packed(seed, [9, 1, 1, 30, 2], (4, 5), 1, late=True)
