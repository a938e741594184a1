"""The memory that the roles of k_packed_attn.cu share, as a model under random schedules (CPU):
test_packed_barriers.py follows the barriers wait by wait, this one what they are there to keep apart.
Every array that one role writes and another reads is a Cell: a write while a reader of the last one
has not come yet is an overwrite, a read of anything but the expected write is a stale or early one.

Held here: planned tiles, marks of missing pages, scales, stages of K and V, queries with their rows'
factors, scores, the warps' maxima and exponents, references' sums, weights and both products' results.
Not held: what one warp keeps for itself between two __syncwarp, and the units' ring (test_paged_barriers.py)."""
import os
import random
import re

import pytest

from conftest import ROOT
from test_paged_barriers import SEEDS, Ring, Schedule, bars

SLOTS = 32


def kernel_source():
    with open(os.path.join(ROOT, "full_duplex_speech_lockstep_gb300", "csrc", "k_packed_attn.cu")) as f:
        return f.read()


def kernel_maxima():
    """Buffers of a group's maxima, as the kernel declares them."""
    m = re.search(r"constexpr int kMaxima = (\d+);", kernel_source())
    return int(m.group(1)) if m else 1


class Cell:
    def __init__(self, name):
        self.name, self.tag, self.left = name, None, 0

    def write(self, tag, readers):
        assert self.left == 0, "%s overwritten: %s by %s, %d still to read" % (
            self.name, self.tag, tag, self.left)
        self.tag, self.left = tag, readers

    def read(self, tag):
        assert self.tag == tag, "%s read of %s, holds %s" % (self.name, tag, self.tag)
        assert self.left > 0, self.name
        self.left -= 1


def cells(name, *shape):
    if not shape:
        return Cell(name)
    return [cells("%s[%d]" % (name, i), *shape[1:]) for i in range(shape[0])]


class Landing:
    """A copy that writes a cell when it lands, or the tensor core's work up to a commit."""

    def __init__(self, what, bar):
        self.what, self.bar = what, bar

    def land(self):
        self.what()
        self.bar.land()

    def arrive(self):
        self.what()
        self.bar.arrive()


class Scales(Landing):
    def land(self):
        self.what()
        self.bar.arrive()


def packed(seed, units, stages, most, buffers=4, maxima=2, together=True, slow=40):
    """Units of so many key tiles in steps of up to `most`.  `maxima`: buffers of the warps' maxima of a
    group; `together`: a half warp has read a planned tile before lane 0 gives it back."""
    s, ring = Schedule(seed), Ring(16)
    ks, vs = stages
    kfull, kempty, vfull, vempty = bars(ks, 17), bars(ks, 1), bars(8, most), bars(vs, 1)
    sfull, sempty = bars(buffers, 2), bars(buffers, 4)
    qfull, qempty = bars(2, 2), bars(2, 8)
    pfull, ofull, oempty = bars(2, 4), bars(2, 1), bars(2, 4)
    tfull, tempty, meet = bars(SLOTS, 1), bars(SLOTS, 2), bars(2, 4)

    tile, missing = cells("tile", SLOTS), cells("missing", SLOTS)
    scales = cells("scales", SLOTS)
    k_stage, v_stage = cells("K stage", ks), cells("V stage", vs)
    query, factor = cells("queries", 2, 2), cells("factors", 2, 2)
    score = cells("scores", buffers)
    top = cells("maxima", 2, maxima, 4)
    total, ref, weight = cells("sums", 2, 4), cells("references", 2), cells("weights", 2, 4)
    product = cells("products", 2)

    edges = {}

    def steps(count):
        return [min(most, count - t) for t in range(0, count, most)]

    first, of_tile = [], []                    # first tile of each step, step of each tile
    for count in units:
        for kt in steps(count):
            first.append(len(of_tile))
            of_tile += [len(first) - 1] * kt
    last_of = {}                               # unit with tiles -> its last step
    at = 0
    for i, count in enumerate(c for c in units if c):
        at += len(steps(count))
        last_of[i] = at - 1

    def planner():
        n = 0
        for k, count in enumerate(units):
            yield from ring.put(k)
            for t in range(count):
                if n >= SLOTS:
                    yield tempty[n % SLOTS], n // SLOTS - 1
                last = t % most == most - 1 or t + 1 == count
                # read by two lanes of either loader's half warp
                tile[n % SLOTS].write((n, most - 1 - t % most if last else -1), 4)
                tfull[n % SLOTS].arrive()
                n += 1
        yield from ring.put(len(units))
        for _ in range(2):
            if n >= SLOTS:
                yield tempty[n % SLOTS], n // SLOTS - 1
            tile[n % SLOTS].write((n, None), 0)
            tfull[n % SLOTS].arrive()
            n += 1

    def late(what):                            # another lane of a half warp
        yield from s.work(slow)
        what()

    def loads(kind, empty):
        n, size, step = 0, len(empty), 0
        while True:
            pair = []
            for m in (n, n + 1):
                yield tfull[m % SLOTS], m // SLOTS
                tag = tile[m % SLOTS].tag
                assert tag[0] == m
                if tag[1] is not None:
                    pair.append(tag)
            for m, _ in pair:
                if m >= size:
                    yield empty[m % size], m // size - 1
            for tag in pair:
                m, lack = tag
                tile[m % SLOTS].read(tag)
                if kind == "k":
                    missing[m % SLOTS].write(m, 4)
                    scales[m % SLOTS].write(None, 0)          # nobody reads the last tile's any more
                    for i in range(16):
                        what = (lambda m=m: scales[m % SLOTS].write(m, 4)) if i == 0 else (lambda: None)
                        s.copies.append(Scales(what, kfull[m % size]))
                    kfull[m % size].expect()
                    s.copies.append(Landing(lambda m=m: k_stage[m % size].write(m, 1), kfull[m % size]))
                else:
                    bar = vfull[step % 8]
                    bar.expect()
                    s.copies.append(Landing(lambda m=m: v_stage[m % size].write(m, 1), bar))
                    for _ in range(max(lack, 0)):
                        bar.arrive()
                step += lack >= 0
                other = lambda m=m, tag=tag: tile[m % SLOTS].read(tag)
                if together:
                    yield from late(other)
                    tempty[m % SLOTS].arrive()
                else:
                    tempty[m % SLOTS].arrive()
                    yield from late(other)
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
                    s.commits.append(Landing(lambda n=n: k_stage[n % ks].read(n), kempty[n % ks]))
                    n += 1
                sfull[step % buffers].arrive()

                def done(step=step, nq=nq):
                    for q in query[nq & 1]:
                        assert q.tag == nq, "queries of another unit"
                        if step == last_of[nq]:
                            q.read(nq)
                    score[step % buffers].write(step, 4)
                s.commits.append(Landing(done, sfull[step % buffers]))
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

                def done(step=step, kt=kt):
                    for m in range(first[step], first[step] + kt):
                        v_stage[m % vs].read(m)
                    for w in weight[step & 1]:
                        w.read(step)
                    product[step & 1].write(step, 4)
                s.commits.append(Landing(done, ofull[step & 1]))
                step += 1
        yield from ring.get(len(units))

    def queries(w):
        nq = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            if not count:
                continue
            if nq >= 2:
                yield qempty[nq & 1], (nq >> 1) - 1
            yield from s.work(6)
            query[nq & 1][w].write(nq, 1)
            factor[nq & 1][w].write(nq, 8)
            qfull[nq & 1].arrive()
            nq += 1
        yield from ring.get(len(units))

    def softmax(g, w):
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
                    buf = (step >> 1) % maxima
                    yield sfull[step % buffers], step // buffers
                    for q in factor[nq & 1]:
                        assert q.tag == nq, "factors of another unit"
                    for m in mine:
                        missing[m % SLOTS].read(m)
                    yield from s.work(5)
                    top[g][buf][w].write(step, 4)
                    meet[g].arrive()
                    yield meet[g], met
                    met += 1
                    yield from s.work(slow)
                    for other in range(4):
                        top[g][buf][other].read(step)
                        yield from s.work(2)
                    if step >= 2:
                        yield oempty[g], (step >> 1) - 1
                    if edges[step] if step in edges else edges.setdefault(step, s.rng.random() < 0.3):
                        yield vfull[step % 8], step // 8
                        for m in mine:
                            assert v_stage[m % vs].tag == m and v_stage[m % vs].left == 1
                    if w == 0:
                        ref[g].write(step, 4)
                    yield from s.work(5)
                    total[g][w].write(step, 4)
                    weight[g][w].write(step, 1)
                    score[step % buffers].read(step)
                    for m in mine:
                        scales[m % SLOTS].read(m)
                    pfull[g].arrive()
                    sempty[step % buffers].arrive()
                step += 1
            for q in factor[nq & 1]:
                q.read(nq)
            qempty[nq & 1].arrive()
            nq += 1
        yield from ring.get(len(units))

    def epilogue(w):
        n = step = 0
        for k, count in enumerate(units):
            yield from ring.get(k)
            for kt in steps(count):
                g = step & 1
                yield pfull[g], step >> 1
                yield from s.work(4)
                ref[g].read(step)
                for t in total[g]:
                    t.read(step)
                yield ofull[g], step >> 1
                yield from s.work(8)
                product[g].read(step)
                oempty[g].arrive()
                for m in range(n, n + kt if w == 0 else n):
                    vempty[m % vs].arrive()
                n += kt
                step += 1
            yield from s.work(10)
        yield from ring.get(len(units))

    s.run([planner(), loads("k", kempty), loads("v", vempty), scores(), values()] +
          [softmax(w // 4, w % 4) for w in range(8)] + [epilogue(w) for w in range(4)] +
          [queries(w) for w in range(2)])


# tiles of a step, buffers of the scores: rows of 2 and 4, of 8, of more, of 32 in fp16
FORMS = [(4, 4), (2, 4), (1, 4), (1, 2)]


@pytest.mark.parametrize("most,buffers", FORMS)
@pytest.mark.parametrize("stages", [(4, 5), (4, 7), (8, 8)])
@pytest.mark.parametrize("seed", SEEDS)
def test_no_role_overwrites_what_another_reads(seed, stages, most, buffers):
    r = random.Random(seed)
    packed(seed, [r.choice([0, 1, 1, 2, 3, 4, 8]) for _ in range(20)], stages, most, buffers,
           kernel_maxima())
    packed(seed, [1] * 25, stages, most, buffers, kernel_maxima())
    packed(seed, [37, 40], stages, most, buffers, kernel_maxima())


@pytest.mark.parametrize("most,buffers", FORMS[:3])
def test_one_buffer_of_maxima_is_written_while_it_is_read(most, buffers):
    with pytest.raises(AssertionError, match="maxima"):
        for seed in range(200):
            packed(seed, [200], (4, 7), most, buffers, maxima=1)


def half_warps_read_together():
    """Whether the loaders' lanes meet between the last read of a planned tile and its return."""
    loader = kernel_source().split("auto load_tiles", 1)[1]
    before = loader.split("mbar_arrive(smem_u32(&ctl->tempty[slot]))", 1)[0]
    return "__syncwarp();" in before.rsplit("load_codes<D>", 1)[1]


@pytest.mark.parametrize("seed", SEEDS)
def test_a_tile_is_given_back_when_all_lanes_have_read_it(seed):
    packed(seed, [100, 1, 3, 90], (4, 7), 4, together=half_warps_read_together())


def test_a_tile_given_back_by_one_lane_alone_is_overwritten():
    with pytest.raises(AssertionError, match="tile"):
        for seed in range(200):
            packed(seed, [200], (4, 7), 4, together=False)
