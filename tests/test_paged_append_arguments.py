"""What the append into bf16 pages takes: arguments that do not fit together are refused, not
read past their ends (CPU); a layer whose queries and keys arrive rotated attends to its
chunks (GPU)."""
import pytest
import torch

import chunk_reference as ref
from sliding_window_gqa_ring_gb300 import carat, engine


def good():
    return dict(key_pages=torch.zeros((6, 128, 2, 256), dtype=torch.bfloat16),
                value_pages=torch.zeros((6, 128, 2, 256), dtype=torch.bfloat16),
                page_table=torch.zeros((3, 2), dtype=torch.int32),
                k_new=torch.zeros((3, 5, 2, 256), dtype=torch.bfloat16),
                v_new=torch.zeros((3, 5, 2, 256), dtype=torch.bfloat16),
                context_lengths=torch.zeros(3, dtype=torch.int32))


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("name,t,error", [
    ("k_new", bf16(3, 5, 1, 256), ValueError), ("k_new", bf16(3, 5, 2, 128), ValueError),
    ("k_new", bf16(3, 5, 512), ValueError), ("v_new", bf16(3, 4, 2, 256), ValueError),
    ("v_new", bf16(2, 5, 2, 256), ValueError), ("v_new", bf16(3, 5, 2, 256).float(), TypeError),
    ("value_pages", bf16(5, 128, 2, 256), ValueError),
    ("value_pages", bf16(6, 128, 2, 256).float(), TypeError),
    ("page_table", torch.zeros((2, 2), dtype=torch.int32), ValueError),
    ("page_table", torch.zeros(6, dtype=torch.int32), ValueError),
    ("page_table", torch.zeros((3, 2), dtype=torch.int64), TypeError),
    ("context_lengths", torch.zeros(2, dtype=torch.int32), ValueError),
    ("context_lengths", torch.zeros(3, dtype=torch.int64), TypeError)])
def test_refusals(name, t, error):
    with pytest.raises(error):
        carat.carat_paged_append(**{**good(), name: t})


def test_a_chunk_of_other_keys_than_queries():
    pool = engine.SharedPool(num_pages=6, page_bytes=128 * 2 * 256 * 2, pages_per_ring=2,
                             device="cpu")
    layer = engine.PagedGlobalLayer(pool, torch.zeros((3, 2), dtype=torch.int32), q_heads=4,
                                    kv_heads=2, head_dim=256, max_chunk=8)
    for batch, k in ((3, 4), (3, 6), (2, 5), (4, 5)):
        with pytest.raises(ValueError, match="k_new of"):
            layer.chunk(bf16(3, 5, 4, 256), bf16(batch, k, 2, 256), bf16(batch, k, 2, 256),
                        torch.zeros(3, dtype=torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("q_heads,kv_heads,head_dim", [(8, 4, 256), (16, 2, 512)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 3)])
def test_chunks_that_arrive_rotated(window, sinks, q_heads, kv_heads, head_dim):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator().manual_seed(60)

    def rows(k, heads):
        return torch.randn((2, k, heads, head_dim), generator=g).bfloat16()

    pool = engine.SharedPool(num_pages=12, page_bytes=128 * kv_heads * head_dim * 2,
                             pages_per_ring=4, fill=float("nan"))
    table = torch.tensor([pool.alloc.alloc_pages(6) for _ in range(2)], dtype=torch.int32).cuda()
    layer = engine.PagedGlobalLayer(pool, table, q_heads=q_heads, kv_heads=kv_heads,
                                    head_dim=head_dim, window=window, sinks=sinks, max_chunk=400)
    keys, values, ctx = rows(0, kv_heads), rows(0, kv_heads), 0
    for k in (400, 123, 1, 4):
        q, kn, vn = rows(k, q_heads), rows(k, kv_heads), rows(k, kv_heads)
        keys, values = torch.cat([keys, kn], 1), torch.cat([values, vn], 1)
        lengths = torch.full((2,), ctx, dtype=torch.int32, device="cuda")
        out = layer.chunk(q.cuda(), kn.cuda(), vn.cuda(), lengths).cpu()
        for b in range(2):
            for j in {0, k // 2, k - 1}:
                want, bound = ref.attention(q[b, j:j + 1].double(), keys[b].double(),
                                            values[b].double(), ctx + j, window, sinks,
                                            layer.scale)
                assert ((out[b, j].double() - want[0]).abs() <= bound[0]).all(), (k, b, j)
        ctx += k
    assert carat.carat_get_device_status(clear=True) == 0
