"""The attention of a chunk over scores far from one another and far from zero, in both of its
forms: CTA pairs, and (few rows of many requests at head_dim 512, wide tables) stream-K (GPU)."""
import pytest
import torch

import chunk_reference as ref
import test_paged_chunk_few_rows_gpu as few
import test_paged_chunk_gpu as base

pytestmark = pytest.mark.gpu
_cuda = base._cuda

PAIRS = [(16, 8, 256, [40, 700], 30), (16, 2, 512, [0, 3700], 3), (4, 2, 512, [300], 140)]
FEW = [(16, 2, 512, [3700] * 16 + [0], 3), (4, 4, 512, [2900] * 9, 4)]
FORMS = [(base.Case, *x) for x in PAIRS] + [(few.Wide, *x) for x in FEW]


@pytest.mark.parametrize("form,q_heads,kv_heads,head_dim,ctx,k", FORMS)
@pytest.mark.parametrize("where", ["all see it", "the last does not"])
def test_a_value_that_is_not_finite_counts_where_its_key_weighs_nothing(
        form, q_heads, kv_heads, head_dim, ctx, k, where):
    """Scores of the first half of the keys lie 260 and more (log2 units) below the others',
    and a key among them has such a value: every query that sees it has it in its output,
    wherever the keys are cut into pieces."""
    window = 0 if where == "all see it" else ctx[-2 if len(ctx) > 1 else 0]
    c = form(ctx, k, q_heads, kv_heads, head_dim, window=window, seed=40)
    c.q[:] = 4.0
    hit = {}
    for b, n in enumerate(ctx):
        low = (n + k) // 2
        c.keys[b][:low] = -1.0
        c.keys[b][low:] = 1.0
        hit[b] = max(0, n + k - 1 - window) if window else n // 7
        if hit[b] < low:
            c.values[b][hit[b], kv_heads - 1, 11] = float("nan")
    c.write()
    got = c.device().call().cpu()
    g = q_heads // kv_heads
    rows = 0
    for b, n in enumerate(ctx):
        for j in range(k):
            sees = hit[b] < (n + k) // 2 and bool(ref.seen(n + j, n + k, window, 0)[hit[b]])
            assert got[b, j, :q_heads - g].isfinite().all(), (b, j)
            if sees:
                assert not got[b, j, q_heads - g:, 11].isfinite().any(), (b, j)
                rows += 1
            else:
                assert got[b, j].isfinite().all(), (b, j)
    assert rows
