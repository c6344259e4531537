"""CPU model of the attention over e4m3 pages, continued: the weights' buffers and the
accumulator under the barriers of test_paged_fp8_schedule_model, and the schedule with
the kernel's own numbers (charge 5, up to 304 ranges, at most 320 pieces a unit) and
requests of fewer queries than proposals."""
import os
import random
import re

import pytest

from test_paged_fp8_schedule_model import KEYS, LAYOUTS, Cta, locate, segments

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "sliding_window_gqa_ring_gb300", "csrc", "paged_fp8_attention.cu")
CHARGE, MAX_PIECES = 5, 320


class Signals(list):
    """The products' signals; the one of a PV product ends its reads."""

    def __init__(self, cta):
        super().__init__()
        self.cta = cta

    def pop(self, i):
        signal = super().pop(i)
        if signal[0] == "o":
            self.cta.weights_read[signal[1] % self.cta.pb] -= 1
            self.cta.products -= 1
        return signal


class WatchedCta(Cta):
    """Counts the PV products that still read a weights' buffer or add to O.  Waits of
    the softmax named in `without` are left out."""

    def __init__(self, *layout, without=()):
        super().__init__(*layout)
        self.weights_read, self.products = [0] * self.pb, 0
        self.queue, self.without = Signals(self), without

    def use(self, kind, g, index):
        if kind == "v":
            # from its first product on; the last one's signal ends it
            self.weights_read[g % self.pb] += 1
            self.products += 1
        yield from super().use(kind, g, index)

    def softmax(self, half):
        for si, g, first, last in self.tiles():
            if first:
                yield self.q_full[si & 1], si >> 1
            yield self.s_full[g & 1], g >> 1
            yield self.sc_full[g % self.slots], g // self.slots
            assert self.scores[g & 1] == g
            # products end in the order they are issued in, QK(g) behind PV(g - 2): with
            # two buffers of weights the wait for that one never has to hold
            assert self.products <= 1
            self.sc_empty[g % self.slots].arrive()
            rescale = not first and random.random() < 0.3
            if self.pb == 2 and g > 1 and "buffer" not in self.without:
                yield self.o_done[g & 1], (g - 2) >> 1
            if g > 0 and (self.pb == 1 and "buffer" not in self.without or
                          rescale and "rescale" not in self.without):
                yield self.o_done[(g - 1) & 1], (g - 1) >> 1
            if rescale:
                assert self.products == 0, "O rescaled under a product"
            assert self.weights_read[g % self.pb] == 0, "weights overwritten under a product"
            w = self.weights[g % self.pb]
            self.weights[g % self.pb] = (g, 1 + (w[1] if w and w[0] == g else 0))
            if last or random.random() < 0.2:      # an edge tile
                yield self.nan_full[si & 1], si >> 1
                if g > 0:
                    yield self.o_done[(g - 1) & 1], (g - 1) >> 1
                for z in range(self.ts):
                    i = self.v_index(g, last) + z
                    yield self.full[i % self.ns], i // self.ns
                    assert self.stage[i % self.ns] == (("v", g, z), True)
                    assert self.reading[i % self.ns] == 0, "V changed under a product"
            self.p_full[g & 1].arrive()
            if last:
                if "output" not in self.without:
                    yield self.o_done[g & 1], g >> 1
                assert self.products == 0 and self.o_of == si, "O read under a product"
                self.written += 1
                self.q_free[si & 1].arrive()


def walk(layout, seed, without=()):
    rng = random.Random(seed)
    random.seed(seed)
    lengths = [rng.choice([1, 1, 2, 3, 9]) for _ in range(rng.randrange(1, 7))]
    cta = WatchedCta(lengths, *LAYOUTS[layout], without=without)
    names = list(cta.roles) + ["land", "tensor"]
    bias = {n: rng.choice([1.0, 1.0, 0.02, 30.0]) for n in names}
    while cta.step(rng, bias):
        pass
    return cta, lengths


@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_no_buffer_changes_under_a_product(layout):
    for seed in range(400):
        cta, lengths = walk(layout, seed)
        assert all(cta.at.get(n) == "end" for n in cta.roles), (seed, lengths, cta.at)
        assert cta.written == len(lengths) * len(cta.soft())
        assert cta.weights_read == [0] * cta.pb and cta.products == 0


# With one buffer of weights every tile waits for the product before it, rescaled or
# not; with two, the wait for the buffer never has to hold (see softmax()).
PLANTED = [(layout, without, fault) for layout in sorted(LAYOUTS)
           for without, fault, buffers in (("buffer", "weights overwritten", (1,)),
                                           ("rescale", "O rescaled", (2,)),
                                           ("output", "O read", (1, 2)))
           if LAYOUTS[layout][2] in buffers]


@pytest.mark.parametrize("layout,without,fault", PLANTED)
def test_the_model_sees_a_missing_wait(layout, without, fault):
    found = set()
    for seed in range(100):
        try:
            walk(layout, seed, without=(without,))
        except AssertionError as e:
            found.add(str(e))
    assert any(fault in f for f in found), found


def kernel_constant(pattern):
    with open(SOURCE) as f:
        return int(re.search(pattern, f.read()).group(1))


def test_the_model_has_the_kernels_numbers():
    assert kernel_constant(r"constexpr int kCharge = (\d+);") == CHARGE
    assert kernel_constant(r"constexpr int kMaxPieces = (\d+);") == MAX_PIECES
    assert kernel_constant(r"constexpr int kKeys = (\d+);") == KEYS


def request_tiles(ctx, n, k, window, capacity):
    if ctx < 0 or not 0 <= n <= k or n > capacity - ctx or n == 0:
        return 0
    first = (ctx - window + 1) // KEYS if window > 0 and ctx >= window else 0
    return (ctx + n - 1) // KEYS - first + 1


@pytest.mark.parametrize("seed", range(400))
def test_the_shipped_schedule_covers_every_tile_once(seed):
    rng = random.Random(1000 + seed)
    batch = rng.choice([1, 1, 2, 3, 8, 31, 33, 64, 130, 400])
    kv_heads, k = rng.choice([1, 2, 8]), rng.randint(1, 16)
    window = rng.choice([0, 0, 1, 100, 128, 1024])
    capacity = rng.choice([256, 4096, 50000])
    tiles = []
    for _ in range(batch):
        n = rng.choice([k, k, rng.randint(0, k), 0, -1, k + 1])
        ctx = rng.choice([-1, 0, capacity - max(n, 0), capacity, rng.randint(0, capacity - k)])
        tiles.append(request_tiles(ctx, n, k, window, capacity))
    # CTAs of the grid over 1 to 4 row groups, one or two CTAs an SM, of 152 and 148 SMs
    ranges = rng.choice([304, 304, 296, 152, 148, 76, 50, 38])
    seen, pieces, table, lasts, at = set(), {}, {}, {}, 0
    for rix in range(ranges):
        st = locate(tiles, kv_heads, ranges, rix, CHARGE)
        assert st["s"] == at
        at = st["e"]
        slots = set()
        for s in segments(st, tiles, kv_heads):
            u = (s["b"], s["c"])
            assert not seen & {(u, x) for x in range(s["x0"], s["x1"])}
            seen |= {(u, x) for x in range(s["x0"], s["x1"])}
            whole = s["x0"] == 0 and s["x1"] == s["n"]
            if s["x0"] == 0:
                table[u] = (rix, -1 if whole else 0 if s["opens"] else 1)
            if s["x1"] == s["n"]:
                lasts[u] = rix
            if not whole:
                slot = 0 if s["opens"] else 1
                assert slot not in slots
                slots.add(slot)
                pieces.setdefault(u, []).append((rix, slot))
    assert at == sum(tiles) * kv_heads == len(seen)
    for b, t in enumerate(tiles):
        for c in range(kv_heads if t else 0):
            assert all(((b, c), x) in seen for x in range(t))
            first, slot = table[(b, c)]
            n = lasts[(b, c)] - first + 1
            if slot < 0:
                assert (b, c) not in pieces and n == 1
            else:
                assert 2 <= n <= MAX_PIECES
                assert pieces[(b, c)] == [(first + q, slot if q == 0 else 0) for q in range(n)]
