"""Host-side argument checks of the attention of a chunk and of the operators on pages
(CPU only: every call fails validation, before any CUDA call), and the pool's shared
pages and compaction plans."""
import math
import os
import random

import pytest

FAKE = 0x10000          # aligned, never dereferenced
MISALIGNED = 0x10008
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def carat():
    from sliding_window_gqa_ring_gb300 import build, carat as c
    if not os.path.exists(c.LIBRARY):
        build.build()
    c.library()
    return c


def _chunk(lib, **kw):
    a = dict(out=FAKE, q=FAKE, kp=FAKE, vp=FAKE, num=8, table=FAKE, mp=4, rows=128, cnt=None,
             ctx=FAKE, k=4, B=2, hq=16, hkv=2, d=512, w=0, s=0, scale=0.1, ws=None, wsb=0,
             stream=None)
    a.update(kw)
    return lib.carat_paged_chunk_attention(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(kp=None), INVALID),
    (dict(vp=None), INVALID), (dict(table=None), INVALID), (dict(ctx=None), INVALID),
    (dict(out=MISALIGNED), INVALID), (dict(q=MISALIGNED), INVALID), (dict(kp=MISALIGNED), INVALID),
    (dict(vp=MISALIGNED), INVALID), (dict(num=0), INVALID), (dict(mp=0), INVALID),
    (dict(rows=0), INVALID), (dict(rows=192), INVALID), (dict(num=1 << 24), INVALID),
    (dict(mp=1 << 24), INVALID), (dict(k=0), INVALID), (dict(k=513), INVALID),
    (dict(B=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(hq=15), INVALID),
    (dict(d=0), INVALID), (dict(w=-1), INVALID), (dict(s=-1), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(d=128), UNSUPPORTED), (dict(hq=130, hkv=2), UNSUPPORTED),
    (dict(B=1 << 26), UNSUPPORTED), (dict(B=0), OK), (dict(B=0, out=None), OK),
])
def test_chunk_checks(carat, kw, status):
    assert _chunk(carat.library(), **kw) == status


@pytest.mark.parametrize("name,least,most", [
    # bytes before and behind `out` (4 x 2 x 16 x 512 bf16 values) that a buffer may begin at
    ("q", 2 * 4 * 16 * 512 * 2, 2 * 4 * 16 * 512 * 2),
    ("kp", 8 * 128 * 2 * 512 * 2, 2 * 4 * 16 * 512 * 2),
    ("vp", 8 * 128 * 2 * 512 * 2, 2 * 4 * 16 * 512 * 2)])
def test_chunk_output_must_not_overlap(carat, name, least, most):
    lib = carat.library()
    at = 1 << 30
    far = dict(out=at, q=at << 1, kp=at << 2, vp=at << 3, ws=at << 4, wsb=1 << 29)
    for there in (at, at + most - 16, at - least + 16):
        assert _chunk(lib, **{**far, name: there}) == INVALID
    need = lib.carat_paged_chunk_workspace_bytes(2, 4, 16, 2, 512)
    assert need == 0 or _chunk(lib, **{**far, "ws": at + most - 16}) == INVALID


HEAD = ("kp", "vp", "ks", "vs", "num", "rows", "row_bytes", "R", "hkv")


def _head(**kw):
    a = dict(kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, num=8, rows=128, row_bytes=512, R=16, hkv=2)
    a.update({x: kw[x] for x in HEAD if x in kw})
    return list(a.values())


def _copy(lib, **kw):
    a = dict(src=FAKE, dst=FAKE, n=None, count=3, stream=None)
    a.update({x: y for x, y in kw.items() if x not in HEAD})
    return lib.carat_pages_copy(*_head(**kw), *a.values())


def _fork(lib, **kw):
    a = dict(table=FAKE, parents_n=4, mp=8, ctx=FAKE, child=2 * FAKE, lens=3 * FAKE, parents=FAKE,
             fresh=FAKE, count=3, stream=None)
    a.update({x: y for x, y in kw.items() if x not in HEAD})
    return lib.carat_paged_fork(*_head(**kw), *a.values())


def _move(lib, **kw):
    a = dict(src=FAKE, dst=FAKE, count=3, table=FAKE, entries=10, stream=None)
    a.update({x: y for x, y in kw.items() if x not in HEAD})
    return lib.carat_pages_move(*_head(**kw), *a.values())


COMMON = [
    (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(kp=MISALIGNED), INVALID),
    (dict(vp=MISALIGNED), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
    (dict(num=0), INVALID), (dict(rows=0), INVALID), (dict(row_bytes=0), INVALID),
    (dict(row_bytes=24), INVALID), (dict(row_bytes=1 << 40), INVALID), (dict(R=0), INVALID),
    (dict(R=48), INVALID), (dict(hkv=0), INVALID), (dict(hkv=1 << 27), INVALID),
    (dict(count=-1), INVALID), (dict(count=0), OK), (dict(count=(1 << 30) + 1), INVALID)]


@pytest.mark.parametrize("call", [_copy, _fork, _move])
@pytest.mark.parametrize("kw,status", COMMON)
def test_page_checks(carat, call, kw, status):
    assert call(carat.library(), **kw) == status


@pytest.mark.parametrize("call,kw,status", [
    (_copy, dict(src=None), INVALID), (_copy, dict(dst=None), INVALID),
    (_copy, dict(kp=None, vp=None), INVALID), (_fork, dict(kp=None, vp=None), INVALID),
    (_move, dict(src=None), INVALID), (_move, dict(dst=None), INVALID),
    (_move, dict(table=None), INVALID), (_move, dict(entries=-1), INVALID),
    (_move, dict(entries=1 << 40), INVALID),
    (_fork, dict(table=None), INVALID), (_fork, dict(child=None), INVALID),
    (_fork, dict(ctx=None), INVALID), (_fork, dict(parents=None), INVALID),
    (_fork, dict(fresh=None), INVALID), (_fork, dict(parents_n=0), INVALID),
    (_fork, dict(mp=0), INVALID), (_fork, dict(mp=1 << 24), INVALID),
    (_fork, dict(child=FAKE), INVALID), (_fork, dict(child=FAKE + 4 * 32 - 4), INVALID),
    (_fork, dict(child=FAKE - 3 * 32 + 4), INVALID), (_fork, dict(lens=FAKE + 12), INVALID),
    (_fork, dict(lens=FAKE - 8), INVALID), (_fork, dict(parents_n=(1 << 30) + 1), INVALID),
])
def test_list_and_table_checks(carat, call, kw, status):
    assert call(carat.library(), **kw) == status


def test_hidden_pages(carat):
    """Against every position that a query at or behind the length sees."""
    for rows in (1, 4, 128):
        for window in (0, 1, 3, 130, 256):
            for sinks in (0, 1, 4, 129):
                for ctx in (0, 1, 2, 5, 127, 128, 129, 300, 1000):
                    first, end = carat.hidden_pages(ctx, window, sinks, rows)
                    assert 0 <= first <= end
                    hidden = set(range(first, end))
                    for page in range(ctx // rows + 2):
                        span = range(page * rows, (page + 1) * rows)
                        seen = not window or any(t > ctx - window or t < sinks for t in span)
                        assert (page in hidden) == (not seen), (rows, window, sinks, ctx, page)


def test_a_shared_page_is_free_when_its_last_owner_gives_it_back(carat):
    pool = carat.Pool(8, 4)
    a = pool.alloc_pages(2)
    assert pool.share_pages([a[0], a[0], a[1]])
    for _ in range(2):
        assert pool.free_pages([a[0]])
    assert pool.stats()["pages"] == 2
    assert not pool.free_pages([a[0], a[0]])            # one owner is left
    assert pool.free_pages([a[0]]) and not pool.free_pages([a[0]])
    assert pool.stats()["pages"] == 1 and pool.stats()["free_pages"] == 7
    assert not pool.share_pages([a[0]]) and not pool.share_pages([a[1], 99])
    assert not pool.share_pages([-1])
    assert pool.free_pages([a[1]]) and pool.free_pages([a[1]])
    assert pool.stats() == {"free_pages": 8, "whole_free_blocks": 2, "rings": 0, "pages": 0}
    # a page that is allocated again has one owner
    b = pool.alloc_pages(8)
    assert pool.free_pages(b) and pool.stats()["pages"] == 0


def test_a_page_of_a_ring_cannot_be_shared(carat):
    pool = carat.Pool(8, 4)
    assert pool.alloc_ring() == 0
    assert not pool.share_pages([0])


def test_compaction_makes_room_for_a_ring(carat):
    pool = carat.Pool(16, 4)
    pages = pool.alloc_pages(16)
    for keep in range(4):                               # one page stays in every block
        assert pool.free_pages([p for p in pages if p // 4 == keep and p % 4 != keep])
    assert pool.alloc_ring() == -1
    assert pool.plan_compaction(0) == ([], [])
    src, dst = pool.plan_compaction(100)
    assert len(src) == len(dst) == 3 and not set(src) & set(dst)
    assert pool.stats() == {"free_pages": 12, "whole_free_blocks": 3, "rings": 0, "pages": 4}
    assert [pool.alloc_ring() for _ in range(4)].count(-1) == 1
    assert pool.plan_compaction(100) == ([], [])


def test_compaction_uses_the_pages_past_the_last_block(carat):
    pool = carat.Pool(10, 4)
    got = pool.alloc_pages(3)
    assert got == [8, 9, 4]
    assert pool.free_pages([9])
    assert pool.plan_compaction(5) == ([4], [9])
    assert pool.stats()["whole_free_blocks"] == 2


@pytest.mark.parametrize("seed", range(20))
def test_random_compactions_keep_every_page(carat, seed):
    """Contents (by name) follow the plan; owners too; nothing is lost or doubled, blocks
    are emptied wholly or not at all, and rings stay where they are."""
    r = random.Random(seed)
    n, ppr = r.choice([(40, 4), (67, 8), (33, 1), (24, 6)])
    pool, held, rings, name = carat.Pool(n, ppr), {}, [], 0
    for _ in range(300):
        what = r.random()
        if what < 0.35:
            for p in pool.alloc_pages(min(r.randint(1, 5), pool.stats()["free_pages"])) or []:
                assert p not in held
                held[p] = [name, 1]
                name += 1
        elif what < 0.6 and held:
            p = r.choice(sorted(held))
            assert pool.free_pages([p])
            held[p][1] -= 1
            if not held[p][1]:
                del held[p]
        elif what < 0.7 and held:
            p = r.choice(sorted(held))
            assert pool.share_pages([p])
            held[p][1] += 1
        elif what < 0.8:
            ring = pool.alloc_ring()
            if ring >= 0:
                rings.append(ring)
        elif what < 0.85 and rings:
            assert pool.free_ring(rings.pop())
        else:
            before = pool.stats()
            budget = r.choice([1, 3, 100])
            src, dst = pool.plan_compaction(budget)
            assert len(src) == len(dst) <= budget
            assert not set(src) & set(dst) and len(set(src)) == len(src)
            assert len(set(dst)) == len(dst) and not set(dst) & set(held)
            for a, b in zip(src, dst):
                assert not any(x // ppr in rings for x in (a, b))
                held[b] = held.pop(a)
            after = pool.stats()
            assert after["pages"] == before["pages"] == len(held)
            assert after["free_pages"] == before["free_pages"]
            assert after["rings"] == before["rings"]
            emptied = {a // ppr for a in src}
            assert after["whole_free_blocks"] == before["whole_free_blocks"] + len(emptied)
    for p, (_, owners) in sorted(held.items()):
        for _ in range(owners):
            assert pool.free_pages([p])
    for ring in rings:
        assert pool.free_ring(ring)
    assert pool.stats()["free_pages"] == n


@pytest.mark.parametrize("table", ["strided", "long", "elsewhere"])
def test_a_table_that_cannot_follow_is_refused_before_pages_are_counted_as_moved(carat, table):
    import types

    import torch

    from sliding_window_gqa_ring_gb300 import engine
    pool = engine.SharedPool(num_pages=8, page_bytes=256, pages_per_ring=4, device="cpu")
    pages = pool.alloc.alloc_pages(8)
    assert pool.alloc.free_pages(pages[1:4] + pages[5:])
    before = pool.alloc.stats()
    bad = {"strided": torch.zeros((2, 8), dtype=torch.int32)[:, ::2],
           "long": torch.zeros((2, 4), dtype=torch.int64),
           "elsewhere": torch.zeros((2, 4), dtype=torch.int32, device="meta")}[table]
    good = types.SimpleNamespace(page_table=torch.zeros((2, 4), dtype=torch.int32))
    with pytest.raises(ValueError):
        pool.compact(iter([good, types.SimpleNamespace(page_table=bad)]), 8)
    assert pool.alloc.stats() == before
    assert pool.alloc.plan_compaction(8)[0]
