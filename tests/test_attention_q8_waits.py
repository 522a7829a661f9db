"""The model of waits (test_attention_waits.py) for the attention over a cache in 8 bits (csrc/attn8_kernel.cuh).

Beside the agents in bf16 a warp fetches the scales of up to two tiles ahead; the issuer of the scores has a part's queries
copied, their units into a ring of four that the softmax reads.
"""
import pytest

from test_attention_waits import PARTS, Model


class Model8(Model):
    ropes = 2                            # places of the rotary boxes

    def producer(self):
        tile = 0
        for part, tiles in enumerate(PARTS):
            for k in range(tiles):
                for g in range(self.groups):
                    n = tile * self.groups + g
                    yield from self.wait(("empty", n % self.slots), n // self.slots - 1)
                    self.copies.append(("full", n % self.slots))
                if self.rotary:
                    yield from self.wait(("x_empty", tile % self.ropes), tile // self.ropes - 1)
                    self.copies.append(("x_full", tile % self.ropes))
                tile += 1

    def scores(self):
        tile = 0
        for part, tiles in enumerate(PARTS):
            yield from self.wait(("q_free",), part - 1)
            self.copies += [("q_full",), ("unit_full", part & 3)]
            yield from self.wait(("q_full",), part)
            for _ in range(tiles):
                yield from self.wait(("s_free", tile & 1), (tile >> 1) - 1)
                for g in range(self.groups if self.latent else 1):
                    n = tile * self.groups + g
                    yield from self.wait(("full", n % self.slots), n // self.slots)
                    if not self.latent:
                        self.products.append(("empty", n % self.slots))
                if self.rotary:
                    yield from self.wait(("x_full", tile % self.ropes), tile // self.ropes)
                    self.products.append(("x_empty", tile % self.ropes))
                self.products.append(("s_full", tile & 1))
                tile += 1
            self.products.append(("q_free",))

    def scales(self):
        for tile in range(sum(PARTS)):
            yield from self.wait(("sc_empty", tile & 1), (tile >> 1) - 1)
            yield
            self.complete(("sc_full", tile & 1))

    def softmax(self):
        tile = 0
        for part, tiles in enumerate(PARTS):
            yield from self.wait(("unit_full", part & 3), part >> 2)
            for k in range(tiles):
                yield from self.wait(("sc_full", tile & 1), tile >> 1)
                self.complete(("sc_empty", tile & 1))
                yield from self.wait(("s_full", tile & 1), tile >> 1)
                self.complete(("s_free", tile & 1))
                if tile > 0 and (tile % 3 == 0 or k == 0):       # reference points that move
                    yield from self.wait(("pv_done",), tile - 1)
                if k == tiles - 1 and not self.latent:
                    n = tile * self.groups + 1
                    yield from self.wait(("full", n % self.slots), n // self.slots)
                if tile > 0:
                    yield from self.wait(("pv_done",), tile - 1)
                self.complete(("p_full",))
                tile += 1
            yield from self.wait(("pv_done",), tile - 1)         # the sums take the weights' place

    def run(self):
        rng = self.rng
        agents = [self.producer(), self.scores(), self.values(), self.softmax(), self.scales()]
        weights = [rng.random() ** 3 + 1e-3 for _ in range(8)]
        idle = 0
        while agents and self.early is None and idle < 20000:
            idle += 1
            if rng.random() < 0.01:
                weights = [rng.random() ** 3 + 1e-3 for _ in range(8)]
            who = rng.choices(range(8), weights)[0]
            if who == 6:
                if self.copies:
                    self.complete(self.copies.pop(rng.randrange(len(self.copies))))
                    idle = 0
            elif who == 7:
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


def runs(slots, groups, latent, rotary, count, ropes=2):
    got = []
    for seed in range(count):
        m = Model8(slots, groups, latent, rotary, seed)
        m.ropes = ropes
        got.append(m.run())
    return sum(e is not None for e, _ in got), sum(stuck for _, stuck in got)


@pytest.mark.parametrize("slots", [4, 6, 8, 10, 12])
def test_grouped(slots):
    assert runs(slots, 2, False, False, 60) == (0, 0)


@pytest.mark.parametrize("ropes", [0, 1, 2])
@pytest.mark.parametrize("slots", [8, 9, 10, 12])
def test_latent(slots, ropes):
    assert runs(slots, 4, True, ropes > 0, 50, ropes) == (0, 0)
