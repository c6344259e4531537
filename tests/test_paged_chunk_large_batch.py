"""The attention of a chunk for as many requests as it takes (refusals on the CPU), and for a
padded batch in which only a few have a token (GPU)."""
import os

import pytest
import torch

import chunk_reference as ref
from sliding_window_gqa_ring_gb300 import build, carat

MOST = 1 << 22
FAKE = 0x10000          # aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not os.path.exists(carat.LIBRARY):
        build.build()
    carat.library()


@pytest.mark.parametrize("head_dim", [256, 512])
def test_more_requests_than_one_call_can_look_through(head_dim):
    def call(batch):
        # (a workspace of no bytes and queries that are not there: neither gets as far as a launch)
        return carat.library().carat_paged_chunk_attention(
            FAKE, None, FAKE, FAKE, 8, FAKE, 4, 128, None, FAKE, 1, batch, 1, 1, head_dim, 0, 0,
            0.1, None, 0, None)
    for batch in (MOST + 1, 1 << 25, 1 << 28):
        assert call(batch) == carat.CARAT_ERR_UNSUPPORTED
        assert carat.paged_chunk_workspace_bytes(batch, 1, 1, 1, head_dim) == 0
    assert call(MOST) == carat.CARAT_ERR_INVALID_ARG
    if head_dim == 512:
        assert carat.paged_chunk_workspace_bytes(MOST, 1, 1, 1, head_dim) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("head_dim", [256, 512])
@pytest.mark.parametrize("k", [1, 3])
def test_a_few_tokens_in_a_large_padded_batch(head_dim, k):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    carat.carat_get_device_status(clear=True)
    batch, q_heads = 1 << 18, 2
    g = torch.Generator().manual_seed(70)
    pages = [torch.randn((64, 128, 1, head_dim), generator=g).bfloat16() for _ in range(2)]
    table = torch.full((batch, 2), -1, dtype=torch.int32)
    lengths = torch.full((batch,), 50, dtype=torch.int32)
    counts = torch.zeros(batch, dtype=torch.int32)
    alive = [0, 7, 31, 32, 4095, batch // 2, batch - 33, batch - 2, batch - 1]
    q = torch.randn((len(alive), k, q_heads, head_dim), generator=g).bfloat16()
    queries = torch.zeros((batch, k, q_heads, head_dim), dtype=torch.bfloat16, device="cuda")
    for i, b in enumerate(alive):
        table[b] = torch.tensor([2 * i, 2 * i + 1])
        lengths[b], counts[b] = 20 * i, 1 + i % k
        queries[b] = q[i].cuda()
    out = torch.full_like(queries, 7.0)
    need = carat.paged_chunk_workspace_bytes(batch, k, q_heads, 1, head_dim)
    carat.carat_paged_chunk_attention(
        out, queries, pages[0].cuda(), pages[1].cuda(), table.cuda(), lengths.cuda(),
        scale=0.0625, new_counts=counts.cuda(),
        workspace=carat.workspace_tensor(need) if need else None)
    assert carat.carat_get_device_status(clear=True) == 0
    for i, b in enumerate(alive):
        n, first = int(counts[b]), int(lengths[b])
        keys, values = (x[2 * i:2 * i + 2].flatten(0, 1)[:first + n].double() for x in pages)
        for j in range(n):
            want, bound = ref.attention(q[i, j:j + 1].double(), keys, values, first + j, 0, 0,
                                        0.0625)
            assert ((out[b, j].cpu().double() - want[0]).abs() <= bound[0]).all(), (b, j)
        out[b, :n] = 7.0
    assert bool((out == 7.0).all())
