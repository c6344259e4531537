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


@pytest.mark.parametrize("seed", range(150))
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
