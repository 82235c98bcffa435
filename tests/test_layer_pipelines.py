"""CPU models of the linear layer's tensor-core pipelines (csrc/linear_tc.cu)
under random interleavings, with the stage, phase and parity arithmetic of the
kernels; barriers and the interleaver are those of test_pipeline_protocols.

  * linear_tc_kernel with CTAS = 2: two CTAs, each with a producer and eight epilogue warps;
    the even CTA's issuer works for both.  "full" lives in the even CTA and
    completes with its expectation and both CTAs' copies; "empty" and
    "accumulator full" exist in each CTA and are completed in both by the
    issuer's commits; "accumulator empty" takes sixteen arrivals.
  * its SPLIT schedule: every K block of every tile belongs to
    exactly one CTA of the tile's cluster, and the closing reduction reads every
    part of every element once.
"""
import random

import pytest

from test_pipeline_protocols import Barrier, interleave


def pair_pipeline(tiles, kblocks, stages, accs, seed, plant=None):
    rng = random.Random(seed)
    full = [Barrier(3, f"full{s}") for s in range(stages)]            # expectation + two copies
    empty = [[Barrier(1, f"empty{c}.{s}") for s in range(stages)] for c in range(2)]
    accf = [[Barrier(1, f"accf{c}.{b}") for b in range(accs)] for c in range(2)]
    acce = [Barrier(16, f"acce{b}") for b in range(accs)]
    ring = [[None] * stages for _ in range(2)]      # slice held by a stage of a CTA
    busy = [[0] * stages for _ in range(2)]         # MMAs still to read it
    acc = [None] * accs                              # tile held by an accumulator
    readers = [set() for _ in range(accs)]
    done = []

    def producer(c):
        g = 0
        for _ in range(tiles):
            for _ in range(kblocks):
                s = g % stages
                if g >= stages and plant != "no empty wait":
                    while not empty[c][s].passed(g // stages - 1):
                        yield
                assert not busy[c][s], "a stage is refilled while an MMA still reads it"
                if c == 0:
                    full[s].arrive()
                    yield
                ring[c][s] = g
                yield
                full[s].arrive()
                g += 1
                yield

    def issuer():
        g = 0
        commits = []
        for i in range(tiles):
            b, u = i % accs, i // accs
            if i >= accs and plant != "no drain wait":
                while not acce[b].passed(u - 1):
                    yield
            assert not readers[b], "an accumulator is refilled while it is drained"
            acc[b] = None
            for _ in range(kblocks):
                s = g % stages
                while not full[s].passed(g // stages + (1 if plant == "full parity" else 0)):
                    yield
                for c in range(2):
                    assert ring[c][s] == g, "an MMA reads another slice"
                    busy[c][s] = 1
                yield
                # the MMA completes, then its commit reaches both CTAs in any order
                commits = [0, 1]
                rng.shuffle(commits)
                for c in range(2):
                    busy[c][s] = 0
                for c in commits:
                    empty[c][s].arrive()
                    yield
                g += 1
            acc[b] = i
            readers[b] = {(c, q) for c in range(2) for q in range(8)}
            for c in (0, 1):
                accf[c][b].arrive()
                yield

    def epilogue(c, q):
        for i in range(tiles):
            b, u = i % accs, i // accs
            while not accf[c][b].passed(u):
                yield
            assert acc[b] == i, "an epilogue warp reads another tile"
            yield
            readers[b].discard((c, q))
            acce[b].arrive()
            yield
        done.append((c, q))

    interleave([producer(0), producer(1), issuer()] +
               [epilogue(c, q) for c in range(2) for q in range(8)], rng)
    assert len(done) == 16


@pytest.mark.parametrize("seed", range(40))
def test_pair_pipeline(seed):
    rng = random.Random(1000 + seed)
    pair_pipeline(rng.randint(1, 7), rng.randint(1, 15), 6, 2, seed)


@pytest.mark.parametrize("seed", range(20))
def test_pair_pipeline_of_single_stages(seed):
    # linear_f32_kernel: two stages, and an accumulator takes one stage
    pair_pipeline(random.Random(2000 + seed).randint(1, 40), 1, 2, 2, seed)


@pytest.mark.parametrize("plant", ["no empty wait", "no drain wait", "full parity"])
def test_pair_pipeline_catches(plant):
    caught = 0
    for seed in range(60):
        try:
            pair_pipeline(12, 1 if plant == "no drain wait" else 9, 6, 2, seed, plant)
        except AssertionError:
            caught += 1
    assert caught > 0


def split_parts(kblocks, size):
    return [(r * kblocks // size, (r + 1) * kblocks // size) for r in range(size)]


@pytest.mark.parametrize("size", [1, 2, 4, 8])
def test_split_covers_k_once(size):
    for kblocks in range(size, 70):
        parts = split_parts(kblocks, size)
        assert [k for a, b in parts for k in range(a, b)] == list(range(kblocks))
        assert all(b > a for a, b in parts)     # a part that is empty would never finish


@pytest.mark.parametrize("bn,threads", [(64, 320), (128, 320)])
def test_split_reduction_reads_every_element_once(bn, threads):
    for rows in (1, 7, 100, 128):
        for size in (1, 2, 4, 8):
            seen = set()
            for rank in range(size):
                for t in range(threads):
                    for i in range(rank * threads + t, rows * (bn // 4), size * threads):
                        assert i not in seen
                        seen.add(i)
            assert seen == set(range(rows * (bn // 4)))


def plane_pipeline(stages_of_k, ring, accs, seed, plant=None):
    """linear_f32_kernel (csrc/linear_f32.cu) with CTAS = 2: a ring of planes,
    three a stage of K in the order 1, 0, 2; the issuer takes them as it needs
    them and releases them in the order 1, 2, 0; an accumulator takes one stage."""
    rng = random.Random(seed)
    full = [Barrier(3, f"full{s}") for s in range(ring)]
    empty = [[Barrier(1, f"empty{c}.{s}") for s in range(ring)] for c in range(2)]
    accf = [[Barrier(1, f"accf{c}.{b}") for b in range(accs)] for c in range(2)]
    acce = [Barrier(16, f"acce{b}") for b in range(accs)]
    held = [[None] * ring for _ in range(2)]    # (stage of K, plane) in a slot of a CTA
    busy = [set() for _ in range(2)]            # slots that an MMA may still read
    acc, readers, done = [None] * accs, [set() for _ in range(accs)], []

    def producer(c):
        g = 0
        for kb in range(stages_of_k):
            for plane in (1, 0, 2):
                s = g % ring
                if g >= ring and plant != "no empty wait":
                    while not empty[c][s].passed(g // ring - 1):
                        yield
                assert s not in busy[c], "a slot is refilled while an MMA still reads it"
                if c == 0:
                    full[s].arrive()
                    yield
                held[c][s] = (kb, plane)
                yield
                full[s].arrive()
                g += 1
                yield

    def issuer():
        g = 0

        def take(kb, plane):
            nonlocal g
            s, u = g % ring, g // ring
            g += 1
            while not full[s].passed(u):
                yield
            for c in range(2):
                assert held[c][s] == (kb, plane), "an MMA reads another plane"
                busy[c].add(s)
            return s

        def commit(s):
            yield
            for c in range(2):
                busy[c].discard(s)
            for c in rng.sample((0, 1), 2):
                empty[c][s].arrive()
                yield

        for kb in range(stages_of_k):
            b, u = kb % accs, kb // accs
            if kb >= accs and plant != "no drain wait":
                while not acce[b].passed(u - 1):
                    yield
            assert not readers[b], "an accumulator is refilled while it is drained"
            acc[b] = None
            s1 = yield from take(kb, 1)
            s0 = yield from take(kb, 0)
            if plant == "early commit":
                yield from commit(s0)
                busy[0].add(s0)
            yield from commit(s1)
            s2 = yield from take(kb, 2)
            yield from commit(s2)
            for c in range(2):
                assert held[c][s0] == (kb, 0), "plane 0 was overwritten"
            if plant != "early commit":
                yield from commit(s0)
            else:
                busy[0].discard(s0)
            acc[b] = kb
            readers[b] = {(c, q) for c in range(2) for q in range(8)}
            for c in (0, 1):
                accf[c][b].arrive()
                yield

    def epilogue(c, q):
        for kb in range(stages_of_k):
            b, u = kb % accs, kb // accs
            while not accf[c][b].passed(u):
                yield
            assert acc[b] == kb, "an epilogue warp reads another stage's sum"
            yield
            readers[b].discard((c, q))
            acce[b].arrive()
            yield
        done.append((c, q))

    interleave([producer(0), producer(1), issuer()] +
               [epilogue(c, q) for c in range(2) for q in range(8)], rng)
    assert len(done) == 16


@pytest.mark.parametrize("ring,accs", [(6, 2), (6, 4), (7, 4), (8, 4)])
@pytest.mark.parametrize("seed", range(10))
def test_plane_pipeline(seed, ring, accs):
    plane_pipeline(random.Random(3000 + seed).randint(1, 30), ring, accs, seed)


@pytest.mark.parametrize("plant", ["no empty wait", "no drain wait", "early commit"])
def test_plane_pipeline_catches(plant):
    caught = 0
    for seed in range(40):
        try:
            plane_pipeline(14, 6, 2, seed, plant)
        except AssertionError:
            caught += 1
    assert caught > 0
