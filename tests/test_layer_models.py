"""CPU models of how the layer operators' launches, pipelines and joins work
together, under random interleavings:

  * what a launch of a chain may read, and where (csrc/layer_math.cuh, chain_begin);
  * linear_tc_kernel's ring with several blocks of K a stage (csrc/linear_tc.cu);
  * linear_f32_kernel's ring of planes with the order in which single CTAs and
    pairs give its slots back (csrc/linear_f32.cu);
  * which thread of which CTA finishes which element of a tile split in K, and
    where in shared memory it finds it (join_parts, csrc/linear_tc.cuh).
"""
import random

import pytest

from test_pipeline_protocols import Barrier, interleave

NEXT, PREV = 1, 2     # kChainNext, kChainPrev


class Launch:
    def __init__(self, name, chain, reads, writes, plain=()):
        """plain: the inputs that are read through the SM's L1 (the others from L2)."""
        self.name, self.chain, self.reads, self.writes, self.plain = name, chain, reads, writes, plain


def backward_calls(kind):
    """The launches of two linear_backward calls on one workspace, each behind one
    that leaves the memory in L1 as it was and one that rewrites the call's inputs
    (csrc/layers_api.cu, linear_backward)."""
    out = []
    for _ in range(2):
        seen = ["X", "W", "dY", "g", "partial"]
        out += [Launch("other use", 0, seen, [], seen),
                Launch("inputs", 0, ["dX", "db"], ["dY", "Z", "X", "W"])]
        if kind == "f32":
            out += [Launch("dz", NEXT, ["dY", "Z"], ["g", "partial"], ["dY", "Z"]),
                    Launch("split", PREV, ["X", "W"], ["xp", "wp"]),
                    Launch("dX", NEXT, ["g", "wp"], ["dX"]),
                    Launch("dW", PREV | NEXT, ["g", "xp"], ["dW"]),
                    Launch("db", PREV, ["partial"], ["db"])]
        elif kind == "16 bits":
            out += [Launch("dz", 0, ["dY", "Z"], ["g", "partial"], ["dY", "Z"]),
                    Launch("dX", NEXT, ["g", "W"], ["dX"]),
                    Launch("dW", PREV | NEXT, ["g", "X"], ["dW"]),
                    Launch("db", PREV, ["partial"], ["db"])]
        else:       # a product in two pieces, whose epilogues read a residual through L1
            out += [Launch("whole waves", NEXT, ["X", "W", "dY"], ["dX"], ["dY"]),
                    Launch("the rest", PREV, ["X", "W", "dY"], ["db"], ["dY"])]
    out.append(Launch("user", 0, ["dX", "db"], ["loss"]))
    return out


def run_chain(launches, seed, plant=None, sms=3, ctas=3):
    """Every CTA of a launch starts once all of the launch before have triggered or
    ended; a wait lasts until the launch before has ended.  An SM's L1 is emptied by
    a wait or a fence alone: nothing promises it to be empty at a launch's start."""
    rng = random.Random(seed)
    l2, l1 = {}, [dict() for _ in range(sms)]
    triggered = [set() for _ in launches]
    ended = [set() for _ in launches]

    def expected(i, name):
        return max((j for j in range(i) if name in launches[j].writes), default=None)

    def cta(i, c, sm):
        x = launches[i]
        plain = x.reads if plant == "through L1" else x.plain

        def wait():
            while i > 0 and len(ended[i - 1]) < ctas:
                yield
            l1[sm].clear()

        if not x.chain & NEXT or plant == "trigger first":
            triggered[i].add(c)
            yield
        if x.chain & PREV:
            if plant not in ("no fence", "through L1"):
                l1[sm].clear()
        else:
            yield from wait()
        triggered[i].add(c)
        yield
        for name in x.reads:
            for part in range(ctas):
                at = (name, part)
                got = l1[sm].get(at, l2.get(at)) if name in plain else l2.get(at)
                if name in plain:
                    l1[sm][at] = got
                assert got == expected(i, name), f"{x.name} reads {name} of launch {got}"
            yield
        for name in x.writes:
            l2[name, c] = i
            l1[sm].pop((name, c), None)
            yield
        if x.chain & PREV and plant != "no wait at the end":
            yield from wait()
        ended[i].add(c)
        triggered[i].add(c)

    live, started = [], 0
    while started < len(launches) or live:
        if started < len(launches) and (started == 0 or len(triggered[started - 1]) == ctas) and \
                rng.random() < 0.3:
            live += [cta(started, c, rng.randrange(sms)) for c in range(ctas)]
            started += 1
        if live:
            g = rng.choice(live)
            try:
                next(g)
            except StopIteration:
                live.remove(g)


KINDS = ["f32", "16 bits", "two pieces"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", range(40))
def test_chained_launches_read_what_was_written(kind, seed):
    run_chain(backward_calls(kind), seed)


@pytest.mark.parametrize("kind,plant", [("f32", "through L1"), ("16 bits", "through L1"),
                                        ("two pieces", "no fence"), ("f32", "trigger first"),
                                        ("16 bits", "trigger first"), ("f32", "no wait at the end"),
                                        ("two pieces", "no wait at the end")])
def test_chained_launches_model_catches(kind, plant):
    caught = 0
    for seed in range(60):
        try:
            run_chain(backward_calls(kind), seed, plant)
        except AssertionError:
            caught += 1
    assert caught > 0


# ------------------------------------------------------------------ rings


class TxBarrier(Barrier):
    """A phase that completes with its one arrival (the expectation) and as many
    copies as were expected; copies may come before the expectation."""

    def __init__(self, name):
        super().__init__(1, name)
        self.copies = 0

    def _check(self):
        if self.pending == 0 and self.copies == 0:
            self.completed += 1
            self.pending = 1

    def expect(self, n):
        assert self.pending == 1, f"{self.name}: expected twice in a phase"
        self.pending = 0
        self.copies += n
        self._check()

    def landed(self):
        self.copies -= 1
        self._check()


def tc_pipeline(ctas, tiles, nk, ks, stages, accs, seed, plant=None):
    """linear_tc_kernel: KS blocks of K a stage, the last stage of a tile with what
    is left; pairs (ctas = 2) with one issuer for both."""
    rng = random.Random(seed)
    full = [TxBarrier(f"full{s}") for s in range(stages)]             # in the even CTA
    empty = [[Barrier(1, f"empty{c}.{s}") for s in range(stages)] for c in range(ctas)]
    accf = [[Barrier(1, f"accf{c}.{b}") for b in range(accs)] for c in range(ctas)]
    acce = [Barrier(8 * ctas, f"acce{b}") for b in range(accs)]
    ring = [[[None] * ks for _ in range(stages)] for _ in range(ctas)]
    busy = [set() for _ in range(ctas)]
    acc, readers, done = [None] * accs, [set() for _ in range(accs)], []

    def producer(c):
        g = 0
        for i in range(tiles):
            for kb in range(0, nk, ks):
                s = g % stages
                if g >= stages and plant != "no empty wait":
                    while not empty[c][s].passed(g // stages - 1):
                        yield
                subs = min(ks, nk - kb)
                if c == 0:
                    full[s].expect(ctas * (ks if plant == "whole stages expected" else subs))
                    yield
                for j in range(subs):
                    assert s not in busy[c], "a stage is refilled while an MMA still reads it"
                    ring[c][s][j] = (i, kb + j)
                    yield
                    full[s].landed()
                    yield
                g += 1

    def issuer():
        g = 0
        for i in range(tiles):
            b, u = i % accs, i // accs
            if i >= accs and plant != "no drain wait":
                while not acce[b].passed(u - 1):
                    yield
            assert not readers[b], "an accumulator is refilled while it is drained"
            acc[b] = []
            for kb in range(0, nk, ks):
                s = g % stages
                while not full[s].passed(g // stages):
                    yield
                for j in range(ks if plant == "whole stages multiplied" else min(ks, nk - kb)):
                    for c in range(ctas):
                        assert ring[c][s][j] == (i, kb + j), "an MMA reads another block of K"
                        busy[c].add(s)
                    acc[b].append(kb + j)
                    yield
                for c in range(ctas):
                    busy[c].discard(s)
                for c in rng.sample(range(ctas), ctas):
                    empty[c][s].arrive()
                    yield
                g += 1
            readers[b] = {(c, q) for c in range(ctas) for q in range(8)}
            for c in range(ctas):
                accf[c][b].arrive()
                yield

    def epilogue(c, q):
        for i in range(tiles):
            b, u = i % accs, i // accs
            while not accf[c][b].passed(u):
                yield
            assert acc[b] == list(range(nk)), "an epilogue warp reads another sum"
            yield
            readers[b].discard((c, q))
            acce[b].arrive()
            yield
        done.append((c, q))

    interleave([producer(c) for c in range(ctas)] + [issuer()] +
               [epilogue(c, q) for c in range(ctas) for q in range(8)], rng, 30000)
    assert len(done) == 8 * ctas


# stages of 227 KB less the epilogue's blocks: 256-wide pairs, 128-wide pairs, 64-wide
RINGS = [(2, 1, 6, 2), (2, 2, 4, 2), (1, 2, 4, 2), (1, 2, 4, 1)]


@pytest.mark.parametrize("ctas,ks,stages,accs", RINGS)
@pytest.mark.parametrize("seed", range(12))
def test_ring_of_stages(ctas, ks, stages, accs, seed):
    rng = random.Random(4000 + seed)
    tiles = 1 if accs == 1 else rng.randint(1, 5)       # (one accumulator: a tile split in K)
    tc_pipeline(ctas, tiles, rng.randint(1, 13), ks, stages, accs, seed)


@pytest.mark.parametrize("plant", ["no empty wait", "no drain wait", "whole stages expected",
                                   "whole stages multiplied"])
def test_ring_of_stages_catches(plant):
    caught = 0
    for seed in range(30):
        try:
            tc_pipeline(2, 6, 1 if plant == "no drain wait" else 9, 2, 4, 2, seed, plant)
        except AssertionError:
            caught += 1
    assert caught > 0


def plane_ring(ctas, stages_of_k, ring, accs, seed, plant=None):
    """linear_f32_kernel: three planes a stage of K in the order 1, 0, 2, multiplied
    as (1,1) (1,0) (0,1) | (2,0) (0,2) (0,0).  Single CTAs give plane 1 back after
    the third product and plane 2 after the fifth, pairs all three at the end.  An
    MMA may read its slots until the next commit has arrived."""
    rng = random.Random(seed)
    full = [TxBarrier(f"full{s}") for s in range(ring)]
    empty = [[Barrier(1, f"empty{c}.{s}") for s in range(ring)] for c in range(ctas)]
    accf = [[Barrier(1, f"accf{c}.{b}") for b in range(accs)] for c in range(ctas)]
    acce = [Barrier(8 * ctas, f"acce{b}") for b in range(accs)]
    held = [[None] * ring for _ in range(ctas)]
    reading = [0] * ring          # MMAs in flight on a slot
    acc, readers, done = [None] * accs, [set() for _ in range(accs)], []

    def producer(c):
        g = 0
        for kb in range(stages_of_k):
            for plane in (1, 0, 2):
                s = g % ring
                if g >= ring and plant != "no empty wait":
                    while not empty[c][s].passed(g // ring - 1):
                        yield
                if c == 0:
                    full[s].expect(ctas)
                    yield
                assert not reading[s], "a slot is refilled while an MMA still reads it"
                held[c][s] = (kb, plane)
                yield
                full[s].landed()
                g += 1
                yield

    def issuer():
        g, flight = 0, []

        def take():
            nonlocal g
            s, u = g % ring, g // ring
            g += 1
            while not full[s].passed(u):
                yield
            return s

        def term(kb, a, pa, b, pb):
            for c in range(ctas):
                assert held[c][a] == (kb, pa) and held[c][b] == (kb, pb), "an MMA reads another plane"
            for s in (a, b):
                reading[s] += 1
                flight.append(s)
            acc[kb % accs].append((pa, pb))
            yield

        def commit(barriers):       # arrives once the MMAs so far have been done
            yield
            while flight:
                reading[flight.pop()] -= 1
            for c in rng.sample(range(ctas), ctas):
                barriers[c].arrive()
                yield

        def release(s):
            yield from commit([empty[c][s] for c in range(ctas)])

        for kb in range(stages_of_k):
            b, u = kb % accs, kb // accs
            if kb >= accs and plant != "no drain wait":
                while not acce[b].passed(u - 1):
                    yield
            assert not readers[b], "an accumulator is refilled while it is drained"
            acc[b] = []
            s1 = yield from take()
            yield from term(kb, s1, 1, s1, 1)
            s0 = yield from take()
            if plant == "plane 1 early":
                yield from release(s1)
            yield from term(kb, s1, 1, s0, 0)
            yield from term(kb, s0, 0, s1, 1)
            if ctas == 1:
                yield from release(s1)
            s2 = yield from take()
            yield from term(kb, s2, 2, s0, 0)
            yield from term(kb, s0, 0, s2, 2)
            if ctas == 1:
                yield from release(s2)
            yield from term(kb, s0, 0, s0, 0)
            if ctas == 2:
                if plant != "plane 1 early":
                    yield from release(s1)
                yield from release(s2)
            yield from release(s0)
            readers[b] = {(c, q) for c in range(ctas) for q in range(8)}
            yield from commit([accf[c][b] for c in range(ctas)])

    def epilogue(c, q):
        for kb in range(stages_of_k):
            b, u = kb % accs, kb // accs
            while not accf[c][b].passed(u):
                yield
            assert sorted(acc[b]) == [(0, 0), (0, 1), (0, 2), (1, 0), (1, 1), (2, 0)]
            yield
            readers[b].discard((c, q))
            acce[b].arrive()
            yield
        done.append((c, q))

    interleave([producer(c) for c in range(ctas)] + [issuer()] +
               [epilogue(c, q) for c in range(ctas) for q in range(8)], rng, 60000)
    assert len(done) == 8 * ctas


@pytest.mark.parametrize("ctas,ring,accs", [(2, 6, 2), (2, 8, 4), (1, 8, 4), (1, 6, 4)])
@pytest.mark.parametrize("seed", range(8))
def test_ring_of_planes(ctas, ring, accs, seed):
    plane_ring(ctas, random.Random(5000 + seed).randint(1, 24), ring, accs, seed)


@pytest.mark.parametrize("plant", ["no empty wait", "no drain wait", "plane 1 early"])
def test_ring_of_planes_catches(plant):
    caught = 0
    for seed in range(30):
        try:
            plane_ring(2, 14, 6, 1 if plant == "no drain wait" else 2, seed, plant)
        except AssertionError:
            caught += 1
    assert caught > 0


# ------------------------------------------------------------------ tiles split in K


def parked(bn):
    """(row, 16-byte chunk of its bn floats) -> first column, as the epilogue warps
    write a part of a tile: warp quarter q, side, 32-column block c, chunk j."""
    at = {}
    for q in range(4):
        for side in range(2):
            for c in range(bn // 64):
                for lane in range(32):
                    r = 32 * q + lane
                    for j in range(8):
                        chunk = side * (bn // 8) + 8 * c + j
                        where = (r, chunk ^ (r & 7))
                        assert where not in at
                        at[where] = 4 * chunk
    return at


@pytest.mark.parametrize("bn", [64, 128, 256])
@pytest.mark.parametrize("parts", [2, 4, 8])
@pytest.mark.parametrize("rows,n", [(128, 512), (128, 37), (77, 250), (1, 512), (9, 64), (0, 512),
                                    (-20, 512)])
def test_join_finishes_every_element_once(bn, parts, rows, n):
    lpr = bn // 8
    rpw = 32 // lpr
    step = 10 * rpw * parts                  # 320 threads
    u_rows = 4 if parts == 2 else 1 if parts == 8 else 2
    at = parked(bn)
    seen = set()
    for part in range(parts):
        for warp in range(10):
            for lane in range(32):
                c = lane % lpr
                col = (4 * c, 4 * (c + lpr))
                if col[0] >= n:
                    continue
                r0 = (warp * parts + part) * rpw + lane // lpr
                while r0 < rows:
                    for u in range(u_rows):
                        r = r0 + u * step
                        if r >= rows:
                            break
                        for h in range(2):
                            chunk = (c + h * lpr) ^ (r & 7)
                            assert at[r, chunk] == col[h]
                            if col[h] < n:
                                for j in range(4):
                                    if col[h] + j < n:
                                        assert (r, col[h] + j) not in seen
                                        seen.add((r, col[h] + j))
                    r0 += u_rows * step
    assert seen == {(r, k) for r in range(max(rows, 0)) for k in range(min(n, bn))}
