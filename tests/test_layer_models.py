"""CPU models of how the layer operators' launches, pipelines and joins work
together, under random interleavings: what a launch of a chain may read, and where
(csrc/layer_math.cuh, chain_begin)."""
import random

import pytest

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
