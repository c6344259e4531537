"""Model of how a CTA pair of the attention of a chunk (csrc/paged_chunk.cu) takes over the work
of clusters that have not been launched, run under random interleavings (CPU only).

The leader asks; the answer lands in both CTAs, each at a moment of its own, at a place that
is used again a few answers later.  Work taken over may be none (a padded batch, rejected
requests): then nothing but the answers goes round.  Checked are, besides what the model of
the other barriers checks, that no answer is written over before it is read, that both CTAs read the
same ones, and that no bytes reach a barrier's phase that expects none of them."""
import os
import random
import re

import pytest

import test_paged_chunk_buffers_model as base
from test_paged_chunk_buffers_model import Barrier, Wrong

SOURCE = os.path.join(base.CSRC, "paged_chunk.cu")


class Taking(base.Pair):
    """units: items (by their tiles' masks) of the pair's own work, then of what it takes over."""

    def __init__(self, units, rng, stages, kst, in_turn, records, jobs, read_first):
        super().__init__([masks for unit in units for masks in unit], rng, stages, kst, in_turn,
                         records, 2, jobs)
        self.units, self.read_first = units, read_first
        both = lambda: [[Barrier(1) for _ in range(jobs)] for _ in range(2)]
        self.answered = both()
        self.answer = [[None] * jobs for _ in range(2)]      # (number, unit or None), unread
        self.answer_read = [Barrier(1) for _ in range(jobs)]   # the leader's

    def ask(self, r, asked):
        """One question; only the leader's makes the answer come."""
        slot = asked % self.jobs
        if self.read_first and r == 0 and asked >= self.jobs:
            while not self.answer_read[slot].passed(asked // self.jobs - 1):
                yield
        self.answered[r][slot].arrive(1)
        if r:
            return
        unit = asked + 1 if asked + 1 < len(self.units) else None
        for to in range(2):
            def land(to=to):
                if self.answer[to][slot] is not None:
                    raise Wrong("an answer is written over before it is read")
                self.answer[to][slot] = (asked, unit)
                if self.answered[to][slot].tx < 0:
                    raise Wrong("two answers' bytes in one phase")
                self.answered[to][slot].land(1)
            self.copy(land)

    def answer_of(self, r, asked):
        slot = asked % self.jobs
        while not self.answered[r][slot].passed(asked // self.jobs):
            yield
        yield
        held = self.answer[r][slot]
        if held is None or held[0] != asked:
            raise Wrong(f"{held} is read for answer {asked}")
        self.answer[r][slot] = None
        if self.read_first and r:
            yield
            self.answer_read[slot].arrive()
        return held[1]

    def producer(self, r):
        cnt = masked_v = asked = j = 0
        unit, pending = 0, False
        while unit is not None:
            for masks in self.units[unit]:
                if j >= self.jobs:
                    while not self.job_empty[r][j % self.jobs].passed(j // self.jobs - 1):
                        yield
                self.job_full[r][j % self.jobs].arrive()
                n = len(masks)
                for x in range(n + 1):
                    loads = [("K", x)] * self.KST if x < n else []
                    if x > 0:
                        loads.append(("V", x - 1))
                    for kind, y in loads:
                        s = cnt % self.NS
                        if cnt >= self.NS:
                            while not self.empty[r][s].passed(cnt // self.NS - 1):
                                yield
                        masked = kind == "V" and masks[y]
                        held, bar = (j, kind, y, cnt), self.full[s]
                        self.stage[r][s] = None
                        if masked:
                            bar = self.v_ready[r][masked_v % self.T]
                            bar.arrive(1)
                            yield
                        if r == 0:
                            self.full[s].arrive(0 if masked else 2)

                        def land(s=s, held=held, bar=bar):
                            self.stage[r][s] = held
                            bar.land(1)
                        yield
                        self.copy(land)
                        cnt += 1
                        masked_v += masked
                    if x == 0:
                        if j > 0:
                            while not self.q_empty[r][0].passed(j - 1):
                                yield
                        if r == 0:
                            self.q_full.arrive(2)
                        self.copy(lambda: self.q_full.land(1))
                        if not pending:
                            yield from self.ask(r, asked)
                            pending = True
                    yield
                j += 1
            if not pending:
                yield from self.ask(r, asked)
            unit = yield from self.answer_of(r, asked)
            asked, pending = asked + 1, False


def units_of(rng):
    """One pair's own work and what it takes over: mostly none, in runs."""
    out = [[masks] for masks in base.items_of(rng)[:2]] if rng.random() < 0.9 else [[]]
    for _ in range(rng.randrange(1, 5)):
        out += [[]] * rng.choice([0, 3, 4, 5, 9, 20])
        out.append(base.items_of(rng)[:rng.choice([0, 1, 1, 2])])
    return out


def runs(seed, which, read_first):
    layouts, in_turn, records, jobs = base.sizes()
    stages, kst = layouts[which]
    for i in range(5):
        rng = random.Random(1000 * seed + i)
        Taking(units_of(rng), rng, stages, kst, in_turn, records, jobs, read_first).run()


def kernel_reads_first():
    """Whether the leader waits until the other CTA has read an answer, and that one says so."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    ask = text[text.index("auto ask = [&]()"):text.index("tc::ask_for_cluster(")]
    rest = text[text.index("tc::cluster_taken("):]
    return (re.search(r"rank == 0 && asked >= kJobs\)\s+alive = warp_wait<true>\("
                      r"&sh->answer_read\[slot\], \(\(asked / kJobs\) & 1\) \^ 1,", ask) is not None
            and re.search(r"rank == 1 && lane == 0\) \{\s+tc::fence_proxy_async_smem\(\);\s+"
                          r"tc::mbar_arrive_cluster\(tc::map_to_rank\(&sh->answer_read\[slot\], 0\)\);",
                          rest) is not None)


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("seed", range(40))
def test_the_kernels_scheme(which, seed):
    runs(seed, which, kernel_reads_first())


@pytest.mark.parametrize("which", [0, 1])
def test_answers_that_nobody_waits_for_are_written_over(which):
    with pytest.raises(Wrong, match="answer"):
        for seed in range(400):
            runs(seed, which, False)
