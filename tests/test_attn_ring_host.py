"""The barriers of the prompts' attention as a model on the host: the loader, the converters (or
the warp that looks values through), the two product warps, the tensor cores and the softmax
warpgroups take steps in random orders, and every wait that a parity lets through is held
against the phase that it meant.  The order of a product warp comes from the kernel's own header."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

STAGES = 5
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "combine_expert_histogram_gb300", "csrc")


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("ring")
    src, lib = str(d / "r.cpp"), str(d / "r.so")
    with open(src, "w") as f:
        f.write('#include "attn_ring.h"\nextern "C" {\n'
                "int tiles(int h, int t, int n) { return ep::ring_tiles(h, t, n); }\n"
                "int before(int h, int t, int n) { return ep::ring_others_before(h, t, n); }\n"
                "int after(int h, int t, int n) { return ep::ring_others_after(h, t, n); }\n}\n")
    subprocess.run([cc, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    return ctypes.CDLL(lib)


class Bar:
    """An mbarrier: phases that are over, arrivals that the present one lacks."""

    def __init__(self, count):
        self.count = self.left = count
        self.over = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left = self.count
            self.over += 1


class Early(Exception):
    """A wait went through whose phase was not the last one to be over."""


class Model:
    """pieces: (halves, tiles) each.  apart: heads of 64 (no turns, S apart from P); fp8: converters;
    two: a loader of keys and one of values.
    skip: a product warp does not wait for the other half's places (as the kernel with turns)."""

    def __init__(self, ring, pieces, apart, fp8, rng, skip=None, two=False):
        self.ring, self.pieces, self.apart, self.fp8, self.rng = ring, pieces, apart, fp8, rng
        self.two, self.skip = two, not apart if skip is None else skip
        self.inside = fp8 and not apart
        n = STAGES
        self.raw_full, self.raw_empty = [Bar(1) for _ in range(n)], [Bar(1) for _ in range(n)]
        self.full, self.empty = [Bar(1 + two) for _ in range(n)], [Bar(2 if fp8 else 3) for _ in range(n)]
        self.q_full, self.s_full, self.s_free, self.o_full, self.turn = ([Bar(1) for _ in range(2)] for _ in range(5))
        self.p_ready = [[Bar(1), Bar(1)] for _ in range(2)]
        self.v_ok = [Bar(1) for _ in range(4)]
        self.published, self.pipe, self.landing = 0, [], []
        self.read = []  # ring places in the order of the products

    # what an actor yields: None (a step of its own), or (barrier, phase): wait until that phase is over
    def loader(self, mine=0):
        n = 0
        empties = self.raw_empty if self.fp8 and not self.inside else self.empty
        for p, (_, nt) in enumerate(self.pieces):
            if mine == 0:
                self.published += 1
            while self.published <= p:
                yield None
            yield None
            for _ in range(2 * nt):
                if n >= STAGES:
                    yield empties[n % STAGES], n // STAGES - 1
                bar = (self.raw_full if self.fp8 else self.full)[n % STAGES]
                if self.two and n % 2 != mine:
                    bar.arrive()
                else:
                    self.landing.append(bar)
                n += 1
                yield None

    def passer(self):
        """Converters, or the warp that looks values through."""
        for n in range(sum(2 * nt for _, nt in self.pieces)):
            s, phase = n % STAGES, n // STAGES
            if self.fp8:
                yield self.raw_full[s], phase
                if not self.inside and n >= STAGES:
                    yield self.empty[s], phase - 1
                self.full[s].arrive()
                if not self.inside:
                    self.raw_empty[s].arrive()
            else:
                yield self.full[s], phase
                if n & 1:
                    self.v_ok[(n >> 1) & 3].arrive()
                self.empty[s].arrive()
            yield None

    def product(self, t):
        base = done = blocks = queries = 0
        for p, (halves, nt) in enumerate(self.pieces):
            while self.published <= p:
                yield None
            mine = self.ring.tiles(halves, t, nt)

            def release(at):
                for _ in range(2 if halves and self.skip else 1):
                    self.pipe.append(self.empty[at % STAGES])

            def walk(at, n):
                for x in range(at, at + n):
                    if not self.skip:
                        yield self.full[x % STAGES], x // STAGES
                        self.empty[x % STAGES].arrive()

            def use(at):
                yield self.full[at % STAGES], at // STAGES
                self.read.append(at)

            at = base
            if mine:
                n = self.ring.before(halves, t, 0)
                yield from walk(at, n)
                at += n
                yield self.q_full[t], queries
                queries += 1
                yield from use(at)
                self.pipe.append(self.s_full[t])
                release(at)
            for i in range(mine):
                yield from use(at + 1)
                if not self.fp8:
                    tile = (at + 1) >> 1
                    if self.rng.random() < 0.5:
                        yield self.v_ok[tile & 3], tile >> 2
                v, more = at + 1, i + 1 < mine
                n = self.ring.before(halves, t, i + 1)
                if self.apart:
                    if more:
                        yield self.s_free[t], done
                        yield from walk(at + 2, n)
                        at += 2 + n
                        yield from use(at)
                        self.pipe.append(self.s_full[t])
                        release(at)
                    yield self.p_ready[t][0], done
                    yield self.p_ready[t][1], done
                    self.pipe.append(self.o_full[t])
                    release(v)
                else:
                    yield self.p_ready[t][0], done
                    if t + blocks:
                        yield self.turn[t], blocks + t - 1
                    yield self.p_ready[t][1], done
                    if more and not self.fp8:
                        yield from walk(at + 2, n)
                        at += 2 + n
                        yield from use(at)
                        self.pipe.append(self.s_full[t])
                    release(v)
                    if more and not self.fp8:
                        release(at)
                    if not more:
                        self.pipe.append(self.o_full[t])
                    if more and self.fp8:
                        yield from walk(at + 2, n)
                        at += 2 + n
                        yield from use(at)
                        self.pipe.append(self.s_full[t])
                        release(at)
                    self.turn[t ^ 1].arrive()
                if not more:
                    at += 2
                done += 1
                blocks += 1
            n = self.ring.after(halves, t, nt)
            yield from walk(at, n)
            assert at + n == base + 2 * nt  # every place was its turn
            if not self.apart and mine < self.ring.tiles(halves, 0, nt):
                yield self.turn[t], blocks + t - 1
                blocks += 1
                self.turn[t ^ 1].arrive()
            base += 2 * nt
            yield None

    def softmax(self, t):
        done = o_done = 0
        for p, (halves, nt) in enumerate(self.pieces):
            while self.published <= p:
                yield None
            mine = self.ring.tiles(halves, t, nt)
            if not mine:
                continue
            self.q_full[t].arrive()
            for i in range(mine):
                yield self.s_full[t], done
                if self.apart:
                    self.s_free[t].arrive()
                    if i:
                        yield self.o_full[t], done - 1
                self.p_ready[t][0].arrive()
                yield None
                self.p_ready[t][1].arrive()
                done += 1
            yield self.o_full[t], done - 1 if self.apart else o_done
            o_done += 1

    def run(self):
        actors = [self.loader(), self.passer(), self.product(0), self.product(1), self.softmax(0), self.softmax(1)]
        if self.two:
            actors.append(self.loader(1))
        state = [next(a, "end") for a in actors]
        slow = self.rng.choice([None, 1, 1, 2, 3, 4, 5])  # an actor that moves late
        idle = 0
        while any(s != "end" for s in state):
            moved = False
            # loads land in any order, products end in theirs
            if self.landing and self.rng.random() < 0.5:
                self.landing.pop(self.rng.randrange(len(self.landing))).arrive()
                moved = True
            if self.pipe and self.rng.random() < 0.5:
                self.pipe.pop(0).arrive()
                moved = True
            x = self.rng.randrange(len(actors))
            if x == slow and self.rng.random() < 0.95:
                x = self.rng.randrange(len(actors))
            s = state[x]
            if s != "end":
                if s is not None:
                    bar, phase = s
                    if bar.over % 2 != phase % 2:  # the parity lets it through
                        if bar.over != phase + 1:
                            raise Early((x, phase, bar.over))
                        moved, state[x] = True, next(actors[x], "end")
                else:
                    moved, state[x] = True, next(actors[x], "end")
            idle = 0 if moved else idle + 1
            assert idle < 20000, "the roles wait for one another"
        return self


def lists(rng):
    """Pieces of a run: rows of few tokens with one tile, or more, between whole row blocks."""
    pieces = []
    for _ in range(rng.randrange(1, 12)):
        nt = rng.choice([0, 1, 1, 1, 2, 2, 3, 4, 5, 7])
        pieces.append((rng.random() < 0.8, nt))
    return pieces


FORMS = [(False, False, False), (False, False, True), (False, True, False), (True, False, False),
         (True, True, False)]


@pytest.mark.parametrize("apart,fp8,two", FORMS)
def test_every_wait_is_for_its_phase(ring, apart, fp8, two):
    rng = random.Random(11)
    for _ in range(400):
        pieces = lists(rng)
        m = Model(ring, pieces, apart, fp8, rng, two=two).run()
        total, base = 0, 0
        for halves, nt in pieces:  # every place read, by one warp or by both
            total += 2 * nt * (1 if halves else 2)
            base += 2 * nt
        assert len(m.read) == total and set(m.read) == set(range(base))


def test_the_shortest_list_that_needs_it(ring):
    """Two row blocks of one tile, then one of two, which the second warp meets without having waited."""
    rng = random.Random(1)
    for _ in range(300):
        Model(ring, [(True, 1), (True, 1), (True, 2)], True, True, rng).run()


def test_the_model_finds_a_wait_without_the_ones_before(ring):
    """A product warp that waits for its own places alone, in a form without turns."""
    rng, found = random.Random(1), 0
    for _ in range(300):
        try:
            Model(ring, [(True, 1), (True, 1), (True, 2)], True, True, rng, skip=True).run()
        except Early:
            found += 1
    assert found > 0
