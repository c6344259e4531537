"""Model of a CTA of the stream-K attention (csrc/attention_tc.cuh): under a window over pages
its softmax looks through the V rows of tiles that not every query sees, and a fused append
writes into a ring's tiles once their V has landed, wherever in a segment such a tile stands.
So its waits for V's stages must not pass on another load's phase (CPU only)."""
import os
import random
import re

import pytest

from test_paged_chunk_buffers_model import CSRC, Barrier, Wrong


class Cta:
    def __init__(self, segments, rng, stages, ks, next_scores=True):
        self.segments, self.rng, self.NS, self.KS = segments, rng, stages, ks
        self.next_scores = next_scores
        self.full = [Barrier(1) for _ in range(stages)]
        self.empty = [Barrier(1) for _ in range(stages)]
        self.s_full = [Barrier(1) for _ in range(2)]
        self.p_full, self.o_done = Barrier(1), Barrier(1)
        self.stage = [None] * stages
        self.events, self.products = [], []

    @staticmethod
    def order(n):
        """K(0), K(x + 1) before V(x), V(n - 1)."""
        parts = [("K", 0)]
        for x in range(n):
            if x + 1 < n:
                parts.append(("K", x + 1))
            parts.append(("V", x))
        return parts

    def producer(self):
        cnt = 0
        for j, masks in enumerate(self.segments):
            for kind, x in self.order(len(masks)):
                for part in range(self.KS):
                    s = cnt % self.NS
                    if cnt >= self.NS:
                        while not self.empty[s].passed(cnt // self.NS - 1):
                            yield
                    self.full[s].arrive(1)

                    def land(s=s, held=(j, kind, x, part)):
                        self.stage[s] = held
                        self.full[s].land(1)
                    self.events.append(land)
                    cnt += 1
                    yield

    def use(self, s, held):
        if self.stage[s] != held:
            raise Wrong(f"a product reads {self.stage[s]} for {held}")

    def issuer(self):
        cnt = g = 0
        for j, masks in enumerate(self.segments):
            n = len(masks)
            for kind, x in self.order(n):
                if kind == "V":
                    while not self.p_full.passed(g + x):
                        yield
                for part in range(self.KS):
                    s = cnt % self.NS
                    while not self.full[s].passed(cnt // self.NS):
                        yield
                    held = (j, kind, x, part)
                    self.products.append(lambda s=s, held=held: self.use(s, held))
                    self.products.append(self.empty[s].arrive)
                    cnt += 1
                    yield
                if kind == "K":
                    self.products.append(self.s_full[(g + x) & 1].arrive)
                else:
                    self.products.append(self.o_done.arrive)
            g += n

    def softmax(self):
        base = g = 0
        for j, masks in enumerate(self.segments):
            n = len(masks)
            for x in range(n):
                tile = g + x
                while not self.s_full[tile & 1].passed(tile >> 1):
                    yield
                yield
                if tile > 0:
                    while not self.o_done.passed(tile - 1):
                        yield
                if masks[x]:
                    if self.next_scores and x + 1 < n:
                        while not self.s_full[(tile + 1) & 1].passed((tile + 1) >> 1):
                            yield
                    at = base + self.order(n).index(("V", x)) * self.KS
                    for part in range(self.KS):
                        while not self.full[(at + part) % self.NS].passed((at + part) // self.NS):
                            yield
                        if self.stage[(at + part) % self.NS] != (j, "V", x, part):
                            raise Wrong("looks through another load")
                yield
                self.p_full.arrive()
            g += n
            base += 2 * n * self.KS

    def run(self):
        roles = [self.producer(), self.issuer(), self.softmax()]
        speed = {id(x): self.rng.choice([1.0, 1.0, 0.2, 0.03]) for x in roles}
        hardware, idle = self.rng.choice([0.05, 0.3, 0.7]), 0
        while roles:
            if self.rng.random() < hardware and (self.events or self.products):
                if self.events and (self.rng.random() < 0.6 or not self.products):
                    self.events.pop(self.rng.randrange(len(self.events)))()
                elif self.products:
                    self.products.pop(0)()
                continue
            role = self.rng.choice(roles)
            if self.rng.random() > speed[id(role)]:
                continue
            try:
                next(role)
            except StopIteration:
                roles.remove(role)
                idle = 0
            idle += 1
            if idle > 400000:
                raise Wrong("waits that never end")


def segments_of(rng):
    return [[rng.random() < 0.5 for _ in range(rng.choice([1, 1, 2, 3, 6]))]
            for _ in range(rng.randrange(2, 6))]


def instantiated():
    """(stages, stages of a tile) of the kernels whose rings are shorter than two tiles."""
    window = open(os.path.join(CSRC, "attention_tc_window.cu")).read()
    found = {(int(x), 4) for x in re.findall(r"launch_tc<512, \d+, (\d+), 1, 0, false, true>",
                                             window)}
    ring = "".join(open(os.path.join(CSRC, f)).read()
                   for f in ("attention_tc.cu", "attention_tc_unit.cu"))
    found |= {(int(x), 2) for x in re.findall(r"launch_tc<256, \d+, (\d+), \d(?:>|, 0, true>)",
                                              ring) if int(x) < 4}
    return sorted(found)


@pytest.mark.parametrize("seed", range(40))
def test_the_kernels_rings(seed):
    assert instantiated() == [(3, 2), (4, 4), (5, 4)]
    for stages, ks in instantiated():
        for i in range(4):
            rng = random.Random(1000 * seed + i)
            Cta(segments_of(rng), rng, stages, ks).run()


@pytest.mark.parametrize("stages,ks", [(3, 2), (4, 4), (5, 4)])
def test_without_the_next_scores_a_wait_passes_too_early(stages, ks):
    with pytest.raises(Wrong):
        for seed in range(4000):
            rng = random.Random(seed)
            Cta(segments_of(rng), rng, stages, ks, next_scores=False).run()
