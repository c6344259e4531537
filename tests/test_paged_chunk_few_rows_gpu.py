"""Few rows of many requests at head_dim 512 whose page tables and windows hold keys enough for
the stream-K form of the attention of a chunk (csrc/attention_tc_window.cu): the cases of
test_paged_chunk_gpu over wide tables, and windows as long (GPU)."""
import os
import re

import pytest
import torch

import chunk_reference as ref
import test_paged_chunk_gpu as base
from sliding_window_gqa_ring_gb300 import carat

pytestmark = pytest.mark.gpu
_cuda = base._cuda

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "sliding_window_gqa_ring_gb300", "csrc", "paged_chunk.cu")
MANY = [(16, 2, 512, 17), (2, 2, 512, 17), (12, 4, 512, 9), (40, 4, 512, 9)]


class Wide(base.Case):
    """The table has as many entries more, of no page, as the rule asks for."""

    def device(self):
        super().device()
        units, tiles = map(int, re.search(r"kStepUnits = (\d+), kStepTiles = (\d+);",
                                          open(SOURCE).read()).groups())
        batch, k, q_heads, _ = self.q.shape
        kv_heads = self.kp.shape[2]
        assert batch * kv_heads >= units and q_heads // kv_heads * k <= 64
        pages = -(-(tiles // (batch * kv_heads) + 1) * 128 // self.page_rows)
        extra = max(0, pages - self.dt.shape[1])
        pad = torch.full((batch, extra), -1, dtype=torch.int32, device="cuda")
        self.dt = torch.cat([self.dt, pad], 1).contiguous()
        seen = self.dt.shape[1] * self.page_rows // 128
        if self.window:
            seen = min(seen, (self.window + k) // 128 + 2 + -(-self.sinks // 128))
        assert batch * kv_heads * seen > tiles
        return self


@pytest.fixture
def wide(monkeypatch):
    monkeypatch.setattr(base, "Case", Wide)


def _ragged(n, longest, seed):
    c = base._ragged(n, longest, seed)
    c[n // 2] = longest - 1111
    return c


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
@pytest.mark.parametrize("k", [1, 3, 4])
@pytest.mark.parametrize("window,sinks", [(0, 0), (513, 1 << 30), (2600, 5), (2433, 0)])
def test_many_requests(q_heads, kv_heads, head_dim, batch, k, window, sinks):
    c = Wide(_ragged(batch, 3700, k), k, q_heads, kv_heads, head_dim, window=window, sinks=sinks,
             seed=20, spread=2.0, page_rows=256).device()
    c.check(c.call())


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
def test_counts(wide, q_heads, kv_heads, head_dim, batch):
    base.test_many_requests_with_counts(q_heads, kv_heads, head_dim, batch, 0)


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
def test_counts_under_a_window(q_heads, kv_heads, head_dim, batch):
    counts = [i % 5 for i in range(batch)]
    c = Wide(_ragged(batch, 3400, 3), 4, q_heads, kv_heads, head_dim, counts=counts, window=2600,
             sinks=130, seed=21).device()
    c.check(c.call())


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
def test_non_finite_values(wide, q_heads, kv_heads, head_dim, batch, bad):
    base.test_non_finite_values_among_many_requests(q_heads, kv_heads, head_dim, batch, 0, bad)


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
@pytest.mark.parametrize("sinks", [0, 2])
def test_non_finite_values_at_both_ends_of_a_window(q_heads, kv_heads, head_dim, batch, sinks):
    """Of each request: the key that leaves the window between the first query and the last,
    one that left it before, and the newest but one; nothing else changes."""
    k, window = 4, 2600
    ctx = [2640 + 9 * i for i in range(batch)]
    clean = Wide(ctx, k, q_heads, kv_heads, head_dim, window=window, sinks=sinks, seed=22)
    c = Wide(ctx, k, q_heads, kv_heads, head_dim, window=window, sinks=sinks, seed=22)
    for b in range(batch):
        c.values[b][ctx[b] + 1 - window, kv_heads - 1, 11] = float("inf")
        c.values[b][ctx[b] - 1 - window, 0, 5] = float("nan")
        c.values[b][ctx[b] + 2, 0, 300] = float("nan")
    c.write()
    got = c.device().call().cpu()
    g = q_heads // kv_heads
    for b in range(batch):
        want, bound = clean.want(b)
        for j in range(k):
            seen = ref.seen(ctx[b] + j, ctx[b] + k, window, sinks)
            for c_head in range(kv_heads):
                hit = (c_head == kv_heads - 1 and bool(seen[ctx[b] + 1 - window]),
                       c_head == 0 and bool(seen[ctx[b] + 2]))
                for h in range(c_head * g, (c_head + 1) * g):
                    if not any(hit):
                        off = (got[b, j, h].double() - want[j, h]).abs()
                        assert (off <= bound[j, h]).all(), (b, j, h)
                    assert not hit[0] or not got[b, j, h, 11].isfinite(), (b, j, h)
                    assert not hit[1] or not got[b, j, h, 300].isfinite(), (b, j, h)


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
def test_some_rejected(wide, q_heads, kv_heads, head_dim, batch):
    base.test_many_requests_some_rejected(q_heads, kv_heads, head_dim, batch)


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY[:2])
def test_bad_pages_queries_and_repeats(wide, q_heads, kv_heads, head_dim, batch):
    base.test_many_requests_bad_pages_queries_and_repeats(q_heads, kv_heads, head_dim, batch)


def test_the_workspace_serves_both_forms():
    """The same call over a narrow and a wide table, one workspace."""
    narrow = base.Case([300] * 17, 2, 16, 2, 512, seed=30).device()
    wide = Wide([300] * 17, 2, 16, 2, 512, seed=30).device()
    wide.ws = narrow.ws
    for c in (narrow, wide, narrow):
        c.out.fill_(7.0)
        c.check(c.call())
    assert carat.carat_get_device_status(clear=True) == 0
