"""A model of every wait of the attention kernel (csrc/attn_kernel.cuh), run in random orders of events on the CPU.

The kernel's warps meet at barriers and tell one use of a place from the next by the parity of a barrier's phase
alone.  A wait by parity for phase n also passes while the barrier is two phases behind, so it is right only where
the waiting warp cannot get there that early.  The model has the kernel's agents (the copy producer, the issuer of
the scores, the issuer of the products with the values, the softmax), its copies that land in any order and its
products that complete in order, and checks at each wait that passes that the phase it means is complete.

A sequence part is a run of tiles with queries of its own; the softmax waits for the values of a part's last tile
itself (where it zeroes the lines behind the end).
"""
import random

import pytest

PARTS = [1, 1, 7, 2, 1, 12, 3, 1, 9]     # tiles of each part


class Model:
    """One run.  latent: `groups` value groups that the scores read too, and a rotary box in a ring of two; grouped:
    a key group and a value group per tile."""

    def __init__(self, slots, groups, latent, rotary, seed):
        self.slots, self.groups, self.latent, self.rotary = slots, groups, latent, rotary
        self.rng = random.Random(seed)
        self.done = {}                   # completed phases per barrier
        self.early = None
        self.copies, self.products = [], []

    def complete(self, bar):
        self.done[bar] = self.done.get(bar, 0) + 1

    def wait(self, bar, phase):
        """Until the barrier's parity says that phase `phase` (from 0) is complete; a fresh barrier's phase -1 is."""
        while (self.done.get(bar, 0) & 1) == (phase & 1):
            yield
        if self.done.get(bar, 0) < phase + 1 and self.early is None:
            self.early = (bar, phase, self.done.get(bar, 0))
        yield

    def producer(self):
        tile = 0
        for part, tiles in enumerate(PARTS):
            for k in range(tiles):
                if part == 0 and k == 0:
                    yield from self.queries(part)
                for g in range(self.groups):
                    n = tile * self.groups + g
                    yield from self.wait(("empty", n % self.slots), n // self.slots - 1)
                    self.copies.append(("full", n % self.slots))
                if self.rotary:
                    yield from self.wait(("x_empty", tile & 1), (tile >> 1) - 1)
                    self.copies.append(("x_full", tile & 1))
                if part > 0 and k == 0:
                    yield from self.queries(part)
                tile += 1

    def queries(self, part):
        yield from self.wait(("q_free",), part - 1)
        self.copies.append(("q_full",))

    def scores(self):
        tile = 0
        for part, tiles in enumerate(PARTS):
            yield from self.wait(("q_full",), part)
            for _ in range(tiles):
                yield from self.wait(("s_free", tile & 1), (tile >> 1) - 1)
                for g in range(self.groups if self.latent else 1):
                    n = tile * self.groups + g
                    yield from self.wait(("full", n % self.slots), n // self.slots)
                    if not self.latent:
                        self.products.append(("empty", n % self.slots))
                if self.rotary:
                    yield from self.wait(("x_full", tile & 1), tile >> 1)
                    self.products.append(("x_empty", tile & 1))
                self.products.append(("s_full", tile & 1))
                tile += 1
            self.products.append(("q_free",))

    def values(self):
        for tile in range(sum(PARTS)):
            yield from self.wait(("p_full",), tile)
            for g in range(0 if self.latent else 1, self.groups):
                n = tile * self.groups + g
                if not self.latent:
                    yield from self.wait(("full", n % self.slots), n // self.slots)
                self.products.append(("empty", n % self.slots))
            self.products.append(("pv_done",))

    def softmax(self):
        tile = 0
        for tiles in PARTS:
            for k in range(tiles):
                yield from self.wait(("s_full", tile & 1), tile >> 1)
                self.complete(("s_free", tile & 1))
                if k == tiles - 1 and not self.latent:
                    n = tile * self.groups + 1
                    yield from self.wait(("full", n % self.slots), n // self.slots)
                if tile > 0:
                    yield from self.wait(("pv_done",), tile - 1)
                self.complete(("p_full",))
                tile += 1
            yield from self.wait(("pv_done",), tile - 1)

    def run(self):
        rng = self.rng
        agents = [self.producer(), self.scores(), self.values(), self.softmax()]
        weights = [rng.random() ** 3 + 1e-3 for _ in range(6)]
        idle = 0
        while agents and self.early is None and idle < 20000:
            idle += 1
            if rng.random() < 0.01:      # now and then somebody else is slow
                weights = [rng.random() ** 3 + 1e-3 for _ in range(6)]
            who = rng.choices(range(6), weights)[0]
            if who == 4:
                if self.copies:
                    self.complete(self.copies.pop(rng.randrange(len(self.copies))))
                    idle = 0
            elif who == 5:
                if self.products:
                    self.complete(self.products.pop(0))
                    idle = 0
            elif who < len(agents):
                try:
                    next(agents[who])
                except StopIteration:
                    agents.pop(who)
                    idle = 0
        return self.early, bool(agents) and self.early is None


def runs(slots, groups, latent, rotary, count):
    got = [Model(slots, groups, latent, rotary, seed).run() for seed in range(count)]
    return sum(e is not None for e, _ in got), sum(stuck for _, stuck in got)


@pytest.mark.parametrize("slots", [4, 6, 8, 10, 12])
def test_grouped_rings_of_an_even_number_of_places(slots):
    assert runs(slots, 2, False, False, 80) == (0, 0)


@pytest.mark.parametrize("rotary", [True, False])
@pytest.mark.parametrize("slots", [8, 9, 10, 11, 12])
def test_latent_rings(slots, rotary):
    assert runs(slots, 4, True, rotary, 60) == (0, 0)


@pytest.mark.parametrize("slots", [3, 5])
def test_the_model_sees_what_an_odd_number_of_places_does(slots):
    """Keys and values then take turns at a place, and a wait for keys can pass on the phase before the values that
    are still to come.  (The launcher refuses such rings.)"""
    early, stuck = runs(slots, 2, False, False, 250)
    assert early > 0
