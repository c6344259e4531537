"""The most workspace that the attention of a chunk asks for, as the header states it, against
what it does ask for, up to the largest sizes it takes (CPU)."""
import os
import random
import re

import pytest

from sliding_window_gqa_ring_gb300 import build, carat

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "carat.h")


def stated():
    """(a, b, c): at most a bytes, or b and c for each request and KV head where that is more."""
    text = open(HEADER).read()
    text = text[text.index("carat_paged_chunk_attention --"):text.index("Operators on pages:")]
    text = re.sub(r"\s*\n \*\s+", " ", text)
    found = re.search(r"at most (\d+) MB, or (\d+) MB and (\d+) bytes for each request and KV head "
                      r"where that is more", text)
    assert found, "the header states no bound, or not in these words"
    return int(found[1]) * 10 ** 6, int(found[2]) * 10 ** 6, int(found[3])


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not os.path.exists(carat.LIBRARY):
        build.build()


def most(batch, kv_heads):
    a, b, c = stated()
    return max(a, b + c * batch * kv_heads)


@pytest.mark.parametrize("head_dim", [256, 512])
@pytest.mark.parametrize("group", [1, 2, 8, 16, 64])
@pytest.mark.parametrize("kv_heads", [1, 3, 8, 1 << 14])
def test_the_largest_calls(head_dim, group, kv_heads):
    for power in range(29):
        for batch in {1 << power, (1 << power) - 1, (1 << 28) // (kv_heads * group)} - {0}:
            k = 1
            while batch * k * kv_heads * group <= 1 << 28:
                need = carat.paged_chunk_workspace_bytes(batch, k, kv_heads * group, kv_heads,
                                                         head_dim)
                assert need <= most(batch, kv_heads), (batch, k)
                k = k * 3 // 2 + 1


def test_random_calls():
    r = random.Random(5)
    large = 0
    for _ in range(20000):
        kv_heads, group = int(2 ** r.uniform(0, 14)), r.choice([1, 2, 3, 5, 8, 16, 40, 64])
        batch = int(2 ** r.uniform(0, 28))
        k = int(2 ** r.uniform(0, 14))
        need = carat.paged_chunk_workspace_bytes(batch, k, kv_heads * group, kv_heads,
                                                 r.choice([256, 512]))
        assert need <= most(batch, kv_heads)
        large += need > 100 << 20
    assert large > 20
