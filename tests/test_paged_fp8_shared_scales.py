"""Layers over e4m3 pages that share pages share their block scales (CPU; the forked
requests' attention on a GPU)."""
import pytest
import torch

from sliding_window_gqa_ring_gb300 import engine


def layer(pool, table, cos_sin, **kw):
    return engine.Fp8PagedLayer(pool, table, cos_sin, q_heads=4, kv_heads=2, head_dim=256,
                                block_rows=32, **kw)


def small(device):
    pool = engine.SharedPool(num_pages=12, page_bytes=128 * 2 * 256 * 2, pages_per_ring=4,
                             device=device)
    return pool, engine.rotary_table(1024, 256, device=device)


def test_scales_by_argument():
    pool, cs = small("cpu")
    table = torch.full((1, 4), -1, dtype=torch.int32)
    one = layer(pool, table, cs)
    assert one.k_scales.shape == (12, 8, 2) and bool((one.k_scales == 1).all())
    assert one.k_scales.data_ptr() != one.v_scales.data_ptr()
    two = layer(pool, table, cs, k_scales=one.k_scales, v_scales=one.v_scales)
    assert two.k_scales is one.k_scales and two.v_scales is one.v_scales


@pytest.mark.parametrize("change", [
    lambda t: None, lambda t: t[:, :4].contiguous(), lambda t: t.double(), lambda t: t.half(),
    lambda t: torch.ones((12, 8, 4))[:, :, ::2], lambda t: t.to("meta"), lambda t: t[:11],
    lambda t: t.flatten()])
def test_scales_that_do_not_fit(change):
    pool, cs = small("cpu")
    table = torch.full((1, 4), -1, dtype=torch.int32)
    good = torch.ones((12, 8, 2))
    for kw in (dict(k_scales=change(good), v_scales=good), dict(k_scales=good, v_scales=change(good))):
        with pytest.raises(ValueError):
            layer(pool, table, cs, **kw)


@pytest.mark.gpu
def test_children_read_their_parents_pages_with_their_scales():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda").manual_seed(50)

    def rows(n, heads, size=1.0):
        return (torch.randn((1, n, heads, 256), generator=g, device="cuda") * size).bfloat16()

    pool, cs = small("cuda")
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    table[0, :2] = torch.tensor(pool.alloc.alloc_pages(2), device="cuda")
    parent = layer(pool, table, cs)
    n = 300
    ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
    parent.append(rows(n, 2, 8.0), rows(n, 2, 40.0), ctx * 0)      # scales of their own
    assert not (parent.v_scales == 1).all()
    child = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    fresh = torch.tensor(pool.alloc.alloc_pages(1), dtype=torch.int32, device="cuda")
    parent.fork(ctx, child, ctx * 0, fresh)
    beam = layer(pool, child, cs, k_scales=parent.k_scales, v_scales=parent.v_scales)
    args = rows(2, 4), rows(2, 2, 8.0), rows(2, 2, 40.0), ctx
    assert torch.equal(beam.step(*args), parent.step(*args))
