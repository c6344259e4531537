"""Model of the barriers between the roles of a CTA pair of the attention of a chunk
(csrc/paged_chunk.cu), run under random interleavings (CPU only).

Every role is a generator that stops wherever the kernel's warp could be overtaken; copies
land and products complete at random later moments.  Checked are: no arrival at a barrier
whose phase has had all of its arrivals, no wait that passes on another phase than its own
(they go by parity), no wait that never ends, no stage overwritten while it is read, and that
the records of values that are not finite are cleared, written and read in that order."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "sliding_window_gqa_ring_gb300", "csrc")
WARPS = 2          # softmax and scanning warps of a CTA that are modelled


class Wrong(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def settle(self):
        if self.pending == 0 and self.tx == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self, tx=0):
        if self.pending == 0:
            raise Wrong("more arrivals than a phase takes")
        self.pending -= 1
        self.tx += tx
        self.settle()

    def land(self, tx):
        self.tx -= tx
        self.settle()

    def passed(self, use):
        """A wait for the completion of phase `use`, by its parity."""
        if (self.phase & 1) == (use & 1):
            return False
        if self.phase != use + 1:
            raise Wrong(f"a wait for phase {use} passed in phase {self.phase}")
        return True


class Pair:
    """items: for each, its tiles' masks."""

    def __init__(self, items, rng, stages, kst, in_turn, records, ahead, jobs=4):
        self.items, self.rng, self.NS, self.KST, self.T = items, rng, stages, kst, in_turn
        self.R, self.ahead, self.jobs = records, ahead, jobs
        both = lambda n, c: [[Barrier(c) for _ in range(n)] for _ in range(2)]
        self.full = [Barrier(1) for _ in range(stages)]
        self.empty = both(stages, 1)
        self.q_full, self.q_empty = Barrier(1), both(1, 1)
        self.s_full, self.pv_done = both(2, 1), both(2, 1)
        self.p_full = [Barrier(2 * WARPS) for _ in range(2)]
        self.v_ready = both(in_turn, 1)
        self.v_clean = [Barrier(2 * WARPS) for _ in range(in_turn)]
        self.job_full = both(jobs, 1)
        self.job_empty = [[Barrier(2 * WARPS + (r == 0)) for _ in range(jobs)] for r in range(2)]
        self.stage = [[None] * stages for _ in range(2)]    # what a stage holds: landed or not
        self.events = []                                    # copies on their way
        self.products = []                                  # issued, in order
        # whose a record is, per CTA; and the items whose output has read it
        self.owner = [list(range(records)) for _ in range(2)]
        self.read = [[0] * WARPS for _ in range(2)]         # items with masked tiles read so far

    # -- what happens by itself
    def copy(self, land):
        self.events.append(land)

    def commit(self, *bars):
        self.products.append(list(bars))

    def step_hardware(self):
        what = self.rng.random()
        if self.events and (what < 0.6 or not self.products):
            self.events.pop(self.rng.randrange(len(self.events)))()
        elif self.products:
            first = self.products[0]
            if callable(first):
                self.products.pop(0)()
            else:
                for bar in first:
                    bar.arrive()
                self.products.pop(0)

    # -- roles
    def producer(self, r):
        cnt = masked_v = 0
        for j, masks in enumerate(self.items):
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
                    held = (j, kind, y, cnt)
                    self.stage[r][s] = None
                    if masked:
                        own = self.v_ready[r][masked_v % self.T]
                        own.arrive(1)
                        yield
                        if r == 0:
                            self.full[s].arrive()
                        bar = own
                    else:
                        bar = self.full[s]
                        if r == 0:
                            bar.arrive(2)

                    def land(r=r, s=s, held=held, bar=bar):
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
                yield

    def take(self, r, j):
        while not self.job_full[r][j % self.jobs].passed(j // self.jobs):
            yield

    def give(self, r, j):
        self.job_empty[r][j % self.jobs].arrive()

    def holds(self, s, held):
        for r in range(2):
            if self.stage[r][s] != held:
                raise Wrong(f"a product reads {self.stage[r][s]} for {held}")

    def issuer(self):
        cnt = g = vcnt = 0
        for j, masks in enumerate(self.items):
            yield from self.take(0, j)
            self.give(0, j)
            n = len(masks)
            while not self.q_full.passed(j):
                yield
            for x in range(n + 1):
                if x < n:
                    for _ in range(self.KST):
                        s = cnt % self.NS
                        while not self.full[s].passed(cnt // self.NS):
                            yield
                        held = (j, "K", x, cnt)
                        self.products.append(lambda s=s, held=held: self.holds(s, held))
                        self.commit(self.empty[0][s], self.empty[1][s])
                        cnt += 1
                        yield
                    buf = (g + x) & 1
                    self.commit(self.s_full[0][buf], self.s_full[1][buf])
                    if x == n - 1:
                        self.commit(self.q_empty[0][0], self.q_empty[1][0])
                if x == 0:
                    continue
                y, s = x - 1, cnt % self.NS
                buf = (g + y) & 1
                while not self.full[s].passed(cnt // self.NS):
                    yield
                if masks[y]:
                    while not self.v_clean[vcnt % self.T].passed(vcnt // self.T):
                        yield
                    vcnt += 1
                while not self.p_full[buf].passed((g + y) >> 1):
                    yield
                held = (j, "V", y, cnt)
                self.products.append(lambda s=s, held=held: self.holds(s, held))
                self.commit(self.empty[0][s], self.empty[1][s])
                self.commit(self.pv_done[0][buf], self.pv_done[1][buf])
                cnt += 1
                yield
            g += n

    def scanner(self, r, w):
        cnt = vcnt = m = 0
        for j, masks in enumerate(self.items):
            yield from self.take(r, j)
            self.give(r, j)
            n, i = len(masks), 0
            for x in range(n):
                if not masks[x]:
                    continue
                while not self.v_ready[r][vcnt % self.T].passed(vcnt // self.T):
                    yield
                at = cnt + (x + 2 if x + 1 < n else n) * self.KST + x
                if self.stage[r][at % self.NS] != (j, "V", x, at):
                    raise Wrong("looks through another tile")
                if w == 0 and i == 0:
                    after = m + self.ahead
                    old = after - self.R
                    if old >= 0 and min(self.read[r]) <= old:
                        raise Wrong("a record is cleared that is still read")
                    self.owner[r][after % self.R] = after
                yield
                for to in range(2):
                    if self.owner[to][m % self.R] != m:
                        raise Wrong("a record is written that is another's")
                yield
                self.v_clean[vcnt % self.T].arrive()
                vcnt += 1
                i += 1
            cnt += n * (self.KST + 1)
            m += i > 0

    def softmax(self, r, w):
        g = m = 0
        for j, masks in enumerate(self.items):
            yield from self.take(r, j)
            for x in range(len(masks)):
                buf = (g + x) & 1
                while not self.s_full[r][buf].passed((g + x) >> 1):
                    yield
                yield
                self.p_full[buf].arrive()
            g += len(masks)
            while not self.pv_done[r][(g - 1) & 1].passed((g - 1) >> 1):
                yield
            if any(masks):
                if self.owner[r][m % self.R] != m:
                    raise Wrong("a record is read that is another's")
                yield
                m += 1
                self.read[r][w] = m
            self.give(r, j)

    def run(self):
        roles = [self.producer(0), self.producer(1), self.issuer()]
        for r in range(2):
            for w in range(WARPS):
                roles += [self.scanner(r, w), self.softmax(r, w)]
        # some are slow
        speed = {id(x): self.rng.choice([1.0, 1.0, 0.2, 0.03]) for x in roles}
        hardware = self.rng.choice([0.05, 0.3, 0.7])
        idle = 0
        while roles:
            if self.rng.random() < hardware and (self.events or self.products):
                self.step_hardware()
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


def items_of(rng):
    out = []
    for _ in range(rng.randrange(3, 9)):
        n = rng.choice([1, 1, 1, 2, 3, 5])
        style = rng.randrange(3)
        if style == 0:
            masks = [False] * max(0, n - 2) + [True] * min(n, 2)
        elif style == 1:
            masks = [True] * n
        else:
            masks = [rng.random() < 0.4 for _ in range(n)]
        out.append(masks)
    return out


def sizes():
    text = open(os.path.join(CSRC, "paged_chunk.cu")).read()
    stages = re.search(r"NS = D == 256 \? (\d+) : (\d+);", text)
    in_turn = re.search(r"constexpr uint32_t kInTurn = (\d+);", text)
    records = re.search(r"constexpr int kRecords = (\d+);", text)
    jobs = re.search(r"constexpr int kJobs = (\d+);", text)
    return ((int(stages[1]), 1), (int(stages[2]), 2)), int(in_turn[1]), int(records[1]), int(jobs[1])


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("seed", range(40))
def test_the_kernels_numbers(which, seed):
    layouts, in_turn, records, jobs = sizes()
    stages, kst = layouts[which]
    for i in range(5):
        rng = random.Random(1000 * seed + i)
        Pair(items_of(rng), rng, stages, kst, in_turn, records, 2, jobs).run()


@pytest.mark.parametrize("in_turn,records,ahead", [(2, 5, 2), (3, 3, 1), (3, 5, 1)])
def test_fewer_are_found_wrong(in_turn, records, ahead):
    with pytest.raises(Wrong):
        for seed in range(4000):
            rng = random.Random(seed)
            Pair(items_of(rng), rng, 4, 1, in_turn, records, ahead).run()
