"""CPU model of the schedule of the attention over e4m3 pages: the ranges the
CTAs cut from the tile sequence, the segments they walk, the unit table and the
order of the loads, against a tile-by-tile count."""
import random

import pytest

KEYS = 128


def request_tiles(ctx, k, window, capacity):
    if ctx < 0 or ctx + k > capacity:
        return 0, 0
    first = (ctx + 1 - window) // KEYS if window > 0 and ctx + 1 > window else 0
    return first, (ctx + k - 1) // KEYS - first + 1


def locate(tiles, kv_heads, ranges, rix, unit_charge):
    """As the kernel's first warp does it, 32 requests a pass."""
    total = sum(tiles) * kv_heads
    units = sum(t > 0 for t in tiles) * kv_heads
    charge = unit_charge if total >= ranges else 0
    cost = total + charge * units
    length = max((cost + ranges - 1) // ranges, charge + 1)
    x0 = rix * length
    x1 = x0 + length if rix + 1 < ranges else cost
    found = {}
    cum_cost = cum_tiles = 0
    for base in range(0, len(tiles), 32):
        if cum_cost > x1:
            break
        lo, tlo = cum_cost, cum_tiles
        for b in range(base, min(base + 32, len(tiles))):
            v = tiles[b]
            per = v + charge
            vc = kv_heads * per if v > 0 else 0
            for which, x in enumerate((x0, x1)):
                if vc > 0 and lo <= x < lo + vc:
                    j = (x - lo) // per
                    r = x - lo - j * per
                    o = 0 if r <= charge else r - charge
                    found[which] = (tlo + j * v + o, b, j, o)
            lo += vc
            tlo += kv_heads * v
        cum_cost, cum_tiles = lo, tlo
    s, b0, c0, off0 = found.get(0, (total, 0, 0, 0))
    e = found[1][0] if 1 in found else total
    return dict(s=s, e=e, b=b0, c=c0, off=off0)


def segments(st, tiles, kv_heads):
    pos, end, b, c, off = st["s"], st["e"], st["b"], st["c"], st["off"]
    n = tiles[b] if pos < end else 0
    while pos < end and off < n:
        ln = min(n - off, end - pos)
        yield dict(b=b, c=c, x0=off, x1=off + ln, n=n, opens=pos == st["s"])
        pos += ln
        off += ln
        if off == n and pos < end:
            off = 0
            c += 1
            if c == kv_heads:
                c, n = 0, 0
                while n == 0 and b + 1 < len(tiles):
                    b += 1
                    n = tiles[b]


@pytest.mark.parametrize("seed", range(400))
def test_every_tile_once_and_every_piece_found(seed):
    rng = random.Random(seed)
    batch = rng.choice([1, 1, 2, 3, 8, 31, 32, 33, 64, 70])
    k, kv_heads = rng.randint(1, 16), rng.choice([1, 2, 8])
    window = rng.choice([0, 0, 1, 100, 128, 1024])
    capacity = rng.choice([256, 4096, 40000])
    ctx = [rng.choice([-1, 0, capacity - k, capacity, rng.randint(0, capacity - k)])
           for _ in range(batch)]
    tiles = [request_tiles(c, k, window, capacity)[1] for c in ctx]
    for c, t in zip(ctx, tiles):
        if 0 <= c <= capacity - k:
            first = request_tiles(c, k, window, capacity)[0]
            lowest = max(0, c + 1 - window) if window else 0
            assert first * KEYS <= lowest < (first + 1) * KEYS
            assert (first + t - 1) * KEYS <= c + k - 1 < (first + t) * KEYS
    ranges = rng.choice([152, 76, 50, 38, 7, 1])
    charge = rng.choice([1, 2, 3])
    seen, pieces, table, lasts, next_s = {}, {}, {}, {}, 0
    for rix in range(ranges):
        st = locate(tiles, kv_heads, ranges, rix, charge)
        assert st["s"] == next_s
        next_s = st["e"]
        segs = list(segments(st, tiles, kv_heads))
        assert sum(s["x1"] - s["x0"] for s in segs) == st["e"] - st["s"]
        partial_slots = set()
        for s in segs:
            u = (s["b"], s["c"])
            for x in range(s["x0"], s["x1"]):
                assert (u, x) not in seen
                seen[(u, x)] = rix
            whole = s["x0"] == 0 and s["x1"] == s["n"]
            if s["x0"] == 0:
                table[u] = (rix, -1 if whole else 0 if s["opens"] else 1)
            if s["x1"] == s["n"]:
                lasts[u] = rix
            if not whole:
                slot = 0 if s["opens"] else 1
                assert slot not in partial_slots
                partial_slots.add(slot)
                pieces.setdefault(u, []).append((rix, slot))
    assert next_s == sum(tiles) * kv_heads
    for b, t in enumerate(tiles):
        for c in range(kv_heads):
            assert all(((b, c), x) in seen for x in range(t))
            if t == 0:
                continue
            first, slot = table[(b, c)]
            n = lasts[(b, c)] - first + 1
            if slot < 0:
                assert (b, c) not in pieces and n == 1
            else:
                assert n >= 2
                assert pieces[(b, c)] == [(first + q, slot if q == 0 else 0) for q in range(n)]
                assert n <= 256


@pytest.mark.parametrize("lengths", [[1], [2], [1, 1, 1], [3, 1, 4], [7], [1, 5]])
@pytest.mark.parametrize("ts", [1, 2])
def test_stage_numbers_of_the_value_tiles(lengths, ts):
    """K of a tile is loaded before V of the one in front of it, except across a
    segment's end, where V comes first; the softmax finds a tile's V stages by
    arithmetic on its number and on whether it ends its segment."""
    firsts = {sum(lengths[:i]) for i in range(len(lengths))}
    total, count, at = sum(lengths), 0, {}
    for g in range(total + 1):
        boundary = g in firsts and g > 0
        for z in range(2):
            is_k = (z == 0) != boundary
            if is_k and g < total:
                at["k", g] = count
                count += ts
            if not is_k and g > 0:
                at["v", g - 1] = count
                count += ts
    ends = {f - 1 for f in firsts if f} | {total - 1}
    for g in range(total):
        assert at["v", g] == ts * (2 * g + (1 if g in ends else 2))


# ---------------------------------------------------------------------------
# The barriers between a CTA's warps, under random interleavings.  A wait for a
# phase is a wait for its parity, so it may mistake an older phase of the same
# parity for its own; every wait here knows the phase it means and checks.

class Barrier:
    def __init__(self, count=1):
        self.count, self.pending, self.tx, self.done = count, count, 0, 0

    def arrive(self, tx=0):
        assert self.pending > 0, "more arrivals than a phase takes"
        self.pending -= 1
        self.tx += tx
        self.flip()

    def land(self, n=1):
        self.tx -= n
        self.flip()

    def flip(self):
        if self.pending == 0 and self.tx == 0:
            self.done += 1
            self.pending = self.count

    def passes(self, phase):
        """A wait for `phase` (0, 1, ...) by its parity; phase -1 passes at once."""
        if (self.done - 1) % 2 != phase % 2:
            return False
        assert self.done >= phase + 1, "an older phase of the same parity"
        return True


class Cta:
    """The kernel's roles as generators that yield the waits they stand at."""

    def __init__(self, lengths, ts, ns, pb, qb, halves, slots=4):
        self.lengths, self.ts, self.ns, self.pb, self.qb, self.slots = lengths, ts, ns, pb, qb, slots
        two = lambda n, c=1: [Barrier(c) for _ in range(n)]
        self.full, self.empty = two(ns), two(ns)
        self.s_full, self.p_full, self.o_done = two(2), two(2, halves), two(2)
        self.q_full, self.q_empty, self.q_free = two(2), two(2), two(2, halves)
        self.nan_full, self.sc_full, self.sc_empty = two(2), two(slots), two(slots, halves)
        self.stage = [None] * ns          # what a stage holds: (load, landed)
        self.scores, self.weights = [None] * 2, [None] * pb
        self.queries, self.factors = [None] * qb, [None] * 2
        self.reading = [0] * ns           # products that still read a stage
        self.o_of = None                  # segment O belongs to
        self.written = 0
        self.flying = []                  # copies in flight
        self.queue = []                   # the products' signals, in order
        self.roles = {"load": self.load(), "scales": self.scales(), "fetch": self.fetch(),
                      "mma": self.mma()}
        for h in range(halves):
            self.roles["soft%d" % h] = self.softmax(h)
        self.at = {}

    def tiles(self):
        g = 0
        for si, n in enumerate(self.lengths):
            for x in range(n):
                yield si, g, x == 0, x + 1 == n
                g += 1

    def k_index(self, g, first):
        return self.ts * (2 * g if first else 2 * g - 1)

    def v_index(self, g, last):
        return self.ts * (2 * g + (1 if last else 2))

    def load(self):
        order, prev = [], None
        for t in list(self.tiles()) + [None]:
            pair = [("k", t), ("v", prev)]
            for kind, tile in pair[::-1] if t and t[2] and prev else pair:
                if tile:
                    order += [(kind, tile[1], z) for z in range(self.ts)]
            prev = t
        for i, what in enumerate(order):
            s = i % self.ns
            if i >= self.ns:
                yield self.empty[s], i // self.ns - 1
            assert self.reading[s] == 0, "a stage overwritten while it is read"
            self.stage[s] = (what, False)
            self.full[s].arrive(tx=1)
            self.flying.append(("stage", s, what))

    def scales(self):
        for _, g, _, _ in self.tiles():
            if g >= self.slots:
                yield self.sc_empty[g % self.slots], g // self.slots - 1
            self.sc_full[g % self.slots].arrive()

    def fetch(self):
        for si in range(len(self.lengths)):
            was = si - self.qb
            if was >= 0:
                yield self.q_empty[was & 1], was >> 1
            if si >= 2:
                yield self.q_free[si & 1], (si - 2) >> 1
            self.queries[si % self.qb] = self.factors[si & 1] = None
            self.q_full[si & 1].arrive(tx=1)
            self.flying.append(("q", si, None))
            self.nan_full[si & 1].arrive()

    def use(self, kind, g, index):
        for z in range(self.ts):
            s = (index + z) % self.ns
            yield self.full[s], (index + z) // self.ns
            assert self.stage[s] == ((kind, g, z), True), "a product reads another load's stage"
            self.reading[s] += 1
            self.queue.append(("free", s))

    def mma(self):
        prev = None
        for t in list(self.tiles()) + [None]:
            pair = [("k", t), ("v", prev)]
            for kind, tile in pair[::-1] if t and t[2] and prev else pair:
                if not tile:
                    continue
                si, g, first, last = tile
                if kind == "k":
                    if first:
                        yield self.q_full[si & 1], si >> 1
                    assert self.queries[si % self.qb] == si
                    self.scores[g & 1] = None
                    yield from self.use("k", g, self.k_index(g, first))
                    self.queue.append(("scores", g))
                    if last:
                        self.queue.append(("q", si))
                else:
                    yield self.p_full[g & 1], g >> 1
                    assert self.weights[g % self.pb] == (g, len(self.soft()))
                    yield from self.use("v", g, self.v_index(g, last))
                    assert first is (self.o_of != si)
                    self.o_of = si
                    self.queue.append(("o", g))
            prev = t

    def soft(self):
        return [r for r in self.roles if r.startswith("soft")]

    def softmax(self, half):
        for si, g, first, last in self.tiles():
            if first:
                yield self.q_full[si & 1], si >> 1
            assert self.factors[si & 1] == si
            yield self.s_full[g & 1], g >> 1
            yield self.sc_full[g % self.slots], g // self.slots
            assert self.scores[g & 1] == g
            self.sc_empty[g % self.slots].arrive()
            if self.pb == 2 and g > 1:
                yield self.o_done[g & 1], (g - 2) >> 1
            if g > 0 and (self.pb == 1 or random.random() < 0.2):
                yield self.o_done[(g - 1) & 1], (g - 1) >> 1
            w = self.weights[g % self.pb]
            assert w is None or w[0] == g or w[0] < g
            self.weights[g % self.pb] = (g, 1 + (w[1] if w and w[0] == g else 0))
            if last or random.random() < 0.2:      # an edge tile
                yield self.nan_full[si & 1], si >> 1
                if g > 0:
                    yield self.o_done[(g - 1) & 1], (g - 1) >> 1
                for z in range(self.ts):
                    i = self.v_index(g, last) + z
                    yield self.full[i % self.ns], i // self.ns
                    assert self.stage[i % self.ns] == (("v", g, z), True)
            self.p_full[g & 1].arrive()
            if last:
                yield self.o_done[g & 1], g >> 1
                assert self.o_of == si
                self.written += 1
                self.q_free[si & 1].arrive()

    def step(self, rng, bias):
        """One random thing that can happen; False when nothing can."""
        can = []
        for name, role in self.roles.items():
            wait = self.at.get(name)
            if wait == "end" or (wait and not wait[0].passes(wait[1])):
                continue
            can.append(("role", name))
        can += [("land", i) for i in range(len(self.flying))]
        can += [("tensor", 0)] if self.queue else []
        if not can:
            return False
        kind, what = rng.choices(can, [bias.get(c[1] if c[0] == "role" else c[0], 1.0)
                                       for c in can])[0]
        if kind == "role":
            try:
                self.at[what] = next(self.roles[what])
            except StopIteration:
                self.at[what] = "end"
        elif kind == "land":
            k, a, b = self.flying.pop(what)
            if k == "stage":
                assert self.stage[a] == (b, False)
                self.stage[a] = (b, True)
                self.full[a].land()
            else:
                self.queries[a % self.qb] = self.factors[a & 1] = a
                self.q_full[a & 1].land()
        else:
            k, a = self.queue.pop(0)
            if k == "free":
                self.reading[a] -= 1
                self.empty[a].arrive()
            elif k == "scores":
                self.scores[a & 1] = a
                self.s_full[a & 1].arrive()
            elif k == "q":
                self.q_empty[a & 1].arrive()
            else:
                self.o_done[a & 1].arrive()
        return True


# (stages of a K tile, ring, weights' buffers, queries' buffers, softmax groups)
LAYOUTS = {"512 x 32": (2, 5, 2, 1, 2), "512 x 16": (2, 6, 2, 1, 2), "512 x 8": (2, 6, 2, 2, 1),
           "256 x 32": (1, 5, 2, 2, 2), "256 x 16": (1, 3, 1, 1, 1), "256 x 8": (1, 3, 1, 2, 1)}


@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_the_warps_never_wait_for_the_wrong_phase(layout):
    for seed in range(400):
        rng = random.Random(seed)
        random.seed(seed)
        lengths = [rng.choice([1, 1, 2, 3, 9]) for _ in range(rng.randrange(0, 7))]
        cta = Cta(lengths, *LAYOUTS[layout])
        names = list(cta.roles) + ["land", "tensor"]
        bias = {n: rng.choice([1.0, 1.0, 0.02, 30.0]) for n in names}
        steps = 0
        while cta.step(rng, bias):
            steps += 1
        assert all(cta.at.get(n) == "end" for n in cta.roles), (seed, lengths, cta.at)
        assert not cta.flying and not cta.queue
        assert cta.written == len(lengths) * len(cta.soft())
