"""A compaction that cannot be carried out is refused before the allocator counts its pages as
moved and before any table is touched (CPU; on a GPU where a device or a stream is needed)."""
import types

import pytest
import torch

from sliding_window_gqa_ring_gb300 import engine


def broken_up(device="cpu", page_bytes=256):
    pool = engine.SharedPool(num_pages=8, page_bytes=page_bytes, pages_per_ring=4, device=device)
    pages = pool.alloc.alloc_pages(8)
    assert pool.alloc.free_pages(pages[1:4] + pages[5:])
    return pool, pages


def layer(device="cpu", **scales):
    table = torch.arange(8, dtype=torch.int32, device=device).view(2, 4)
    return types.SimpleNamespace(page_table=table, **scales)


def refused(pool, layers, match, **kw):
    before = pool.alloc.stats()
    tables = [x.page_table.clone() for x in layers]
    with pytest.raises(ValueError, match=match):
        pool.compact(layers, 8, **kw)
    assert pool.alloc.stats() == before
    assert all(torch.equal(x.page_table, t) for x, t in zip(layers, tables))


GOOD = torch.ones((8, 2, 3))


@pytest.mark.parametrize("k,v", [
    (GOOD, None), (None, GOOD), (GOOD.double(), GOOD.double()), (GOOD, GOOD.half()),
    (torch.ones((8, 2, 6))[:, :, ::2], GOOD), (GOOD, torch.ones((8, 2, 6))[:, :, ::2]),
    (GOOD, torch.ones((8, 3, 2))), (torch.ones((7, 2, 3)), torch.ones((7, 2, 3))),
    (torch.ones((8, 6)), torch.ones((8, 6))), (GOOD.to("meta"), GOOD.to("meta")),
    (GOOD, GOOD.to("meta"))])
def test_scales_that_cannot_follow(k, v):
    pool, _ = broken_up()
    refused(pool, [layer(), layer(k_scales=k, v_scales=v)], "block scales")
    assert pool.alloc.plan_compaction(8)[0]


def test_pages_of_odd_sizes():
    refused(broken_up(page_bytes=250)[0], [layer()], "16 bytes")


def test_a_pool_on_the_host():
    refused(broken_up()[0], [layer(), layer(k_scales=GOOD, v_scales=GOOD)], "current CUDA device")


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["current", "given", "current, another given"])
def test_streams_under_capture_and_what_is_no_stream(where):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pool, pages = broken_up("cuda")
    one = layer("cuda")
    other = torch.cuda.Stream()
    refused(pool, [one], "invalid literal", stream="nothing")
    graph, captured = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    kept = torch.zeros(4, device="cuda")
    before, table = pool.alloc.stats(), one.page_table.tolist()
    torch.cuda.synchronize()
    with torch.cuda.stream(captured):
        graph.capture_begin(capture_error_mode="thread_local")
        kept.add_(1)
        if where == "given":
            with torch.cuda.stream(other), pytest.raises(ValueError, match="captured"):
                pool.compact([one], 8, stream=captured)
        else:
            with pytest.raises(ValueError, match="captured"):
                pool.compact([one], 8, stream=None if where == "current" else other)
        graph.capture_end()
    graph.replay()
    torch.cuda.synchronize()
    assert kept.tolist() == [1, 1, 1, 1]
    assert pool.alloc.stats() == before and one.page_table.tolist() == table
    # and then it goes ahead
    moved = pool.compact([one], 8, stream=other)
    torch.cuda.synchronize()
    assert moved == 1 and one.page_table.tolist() != table
