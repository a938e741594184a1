"""The barrier protocol of k_packed_attn.cu as a model, under random schedules (CPU): see
test_paged_barriers.py, whose barriers and schedules these are.  The roles follow the kernel wait by
wait; a change to its barriers belongs here first."""
import random

import pytest

from test_paged_barriers import SEEDS, Bar, Ring, Schedule, bars  # noqa: F401


def packed(seed, units, stages, late=False):
    """Units of (key tiles, whether tiles are edges).  `late`: the softmax reuses the weights' buffer as
    soon as its product is done, before the epilogue has taken the tile's sums."""
    s, ring = Schedule(seed), Ring(15)
    kfull, kempty = bars(stages, 1), bars(stages, 4)
    vfull, vempty = bars(stages, 1), bars(stages, 4)
    qfull, qempty = bars(2, 1), bars(2, 8)
    sfull, pfull, ofull, oempty = bars(2, 1), bars(2, 4), bars(2, 1), bars(2, 4)
    meet = bars(2, 4)

    def tiles(full, empty, unit):
        n = 0
        for k, count in enumerate(units):
            yield from unit(k)
            for _ in range(count):
                if n >= stages:
                    yield empty[n % stages], n // stages - 1
                s.load(full[n % stages])
                n += 1
        yield from unit(len(units))

    def issuer():
        n = nq = 0

        def values(m):
            yield pfull[m & 1], m >> 1
            yield vfull[m % stages], m // stages
            s.commits.append(ofull[m & 1])
        k = left = 0
        fresh = True
        while True:                             # step n: values of tile n - 2, scores of tile n
            fresh = left == 0
            while left == 0 and k <= len(units):
                yield from ring.get(k)
                left = units[k] if k < len(units) else 0
                k += 1
            if n >= 2:
                yield from values(n - 2)
            if left == 0:
                break
            if fresh:
                yield qfull[nq & 1], nq >> 1
            yield kfull[n % stages], n // stages
            s.commits.append(sfull[n & 1])
            n, left = n + 1, left - 1
            nq += left == 0
        if n >= 1:
            yield from values(n - 1)

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
        n = nq = met = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            if not count:
                continue
            yield qfull[nq & 1], nq >> 1
            for _ in range(count):
                if (n & 1) == g:
                    yield sfull[g], n >> 1
                    yield kfull[n % stages], n // stages
                    kempty[n % stages].arrive()
                    yield from s.work(5)
                    yield vfull[n % stages], n // stages
                    meet[g].arrive()
                    yield meet[g], met
                    met += 1
                    if n >= 2:
                        if late:
                            yield ofull[g], (n >> 1) - 1
                        else:
                            yield oempty[g], (n >> 1) - 1
                    yield from s.work(5)
                    pfull[g].arrive()
                n += 1
            qempty[nq & 1].arrive()
            nq += 1
        yield from ring.get(len(units))

    def epilogue():
        n = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            for _ in range(count):
                yield pfull[n & 1], n >> 1
                yield ofull[n & 1], n >> 1
                yield from s.work(8)
                oempty[n & 1].arrive()
                vempty[n % stages].arrive()
                n += 1
            yield from s.work(10)
        yield from ring.get(len(units))

    s.run([tiles(kfull, kempty, ring.put), tiles(vfull, vempty, ring.get), issuer(), queries()] +
          [softmax(w // 4) for w in range(8)] + [epilogue() for _ in range(4)])


@pytest.mark.parametrize("stages", [4, 5, 8])
@pytest.mark.parametrize("seed", SEEDS)
def test_packed_attention(seed, stages):
    r = random.Random(seed)
    packed(seed, [r.choice([0, 1, 1, 2, 3, 4, 8]) for _ in range(30)], stages)
    packed(seed, [r.choice([0, 1, 1, 2]) for _ in range(60)], stages)
    packed(seed, [1] * 40, stages)


def test_a_buffer_that_is_used_again_too_early_mistakes_a_phase():
    with pytest.raises(AssertionError, match="phase|deadlock"):
        for seed in range(200):
            packed(seed, [9, 1, 1, 30, 2], 5, late=True)
