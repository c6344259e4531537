"""carat_global_verify_attention_paged over pages whose every other byte is a NaN: what
lies behind a request's keys, in its last page or in pages of nobody, never counts
(GPU, against 64 bits)."""
import pytest
import torch

import paged_reference as ref
from sliding_window_gqa_ring_gb300 import carat, engine

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    carat.library()
    carat.carat_get_device_status(clear=True)
    yield
    assert carat.carat_get_device_status(clear=True) == 0


@pytest.mark.parametrize("keys", [[4, 127, 128, 129], [1000], [300, 255, 257, 512, 640, 4]])
@pytest.mark.parametrize("k,q_heads,kv_heads,head_dim", [(1, 16, 8, 256), (4, 16, 2, 512),
                                                         (4, 64, 2, 512)])
@pytest.mark.parametrize("page_rows", [128, 256])
def test_stale_nans_never_count(keys, k, q_heads, kv_heads, head_dim, page_rows):
    B = len(keys)
    per = -(-max(keys) // page_rows)
    pool = engine.SharedPool(num_pages=B * per + 4, page_bytes=page_rows * kv_heads * head_dim * 2,
                             pages_per_ring=4, fill=float("nan"))
    table = torch.tensor([pool.alloc.alloc_pages(per) for _ in range(B)], dtype=torch.int32)
    cs = engine.rotary_table(per * page_rows, head_dim)
    layer = engine.PagedGlobalLayer(pool, table.cuda(), q_heads=q_heads, kv_heads=kv_heads,
                                    head_dim=head_dim, max_proposals=k, cos_sin=cs)
    g = torch.Generator().manual_seed(81)

    def rows(n, h):
        return torch.randn((B, n, h, head_dim), generator=g).bfloat16().cuda()

    have = [n - k for n in keys]
    ctx = torch.tensor(have, dtype=torch.int32, device="cuda")
    most = max(1, max(have))
    layer.append(rows(most, kv_heads), rows(most, kv_heads), torch.zeros_like(ctx), new_counts=ctx)
    out = layer.step(rows(k, q_heads), rows(k, kv_heads), rows(k, kv_heads), ctx).cpu().double()
    assert carat.carat_get_device_status(clear=True) == 0
    turned = layer.rotated.view(B, k, q_heads, head_dim).cpu().double()
    for b, n in enumerate(keys):
        kk, vv = (p.cpu()[table[b].long()].flatten(0, 1)[:n].double()
                  for p in (layer.key_pages, layer.value_pages))
        want, weight = ref.attention(turned[b], kk, vv, [n - k + j for j in range(k)], 0,
                                     layer.scale)
        # weights rounded to bf16 (2^-8), scores accumulated in fp32
        a = ref.score_magnitude(turned[b], kk, layer.scale)
        tol = 2 * (2.0 ** -8 + a * (head_dim + 64) * 2.0 ** -24) * weight + 2.0 ** -20 * want.abs()
        assert ((out[b] - want).abs() <= tol).all(), b
