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


@pytest.mark.parametrize("form,q_heads,kv_heads,head_dim,ctx,k", FORMS)
@pytest.mark.parametrize("power", [9, 16, 24, 40, 56])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_large_scores(form, q_heads, kv_heads, head_dim, ctx, k, power, sign):
    """Queries and keys of 2^power: scores of about 2^(2 power + 5), of which the products'
    fp32 sums hold some 24 bits.  Where the largest lies further above the others than that
    rounding, (D + 64) 2^-24 of scale sum |q k|, the softmax is one-hot and the output its
    value, rounded twice to bf16 with its weight; no row may be anything but a number."""
    c = form(ctx, k, q_heads, kv_heads, head_dim, scale=sign, seed=41)
    c.q = (c.q.float() * 2.0 ** power).bfloat16()
    for x in c.keys:
        x[:] = (x.float() * 2.0 ** power).bfloat16()
    c.write()
    got = c.device().call().cpu()
    assert got.isfinite().all()
    g, compared = q_heads // kv_heads, 0
    for b, n in enumerate(ctx):
        for j in range(k):
            for h in range(q_heads):
                q = c.q[b, j, h].double()
                keys = c.keys[b][:n + j + 1, h // g].double()
                s = sign * (keys @ q)
                off = float((keys.abs() @ q.abs()).max()) * (head_dim + 64) * 2.0 ** -24
                top = s.topk(min(2, len(s))).values
                if len(s) == 1 or top[0] - top[1] > 2 * off + 40:
                    want = c.values[b][int(s.argmax()), h // g].double()
                    size = 2.0 ** -7 * want.abs() + 2.0 ** -30
                    assert ((got[b, j, h].double() - want).abs() <= size).all(), (b, j, h)
                    compared += 1
    assert compared > sum(1 for _ in ctx) * k


@pytest.mark.parametrize("form,q_heads,kv_heads,head_dim,ctx,k", FORMS)
@pytest.mark.parametrize("scale", [0.0, 1e-40, -1e-40])
def test_scales_of_next_to_nothing_over_large_scores(form, q_heads, kv_heads, head_dim, ctx, k,
                                                     scale):
    """Scores of about 2^123 times 1e-40 are below 2^-7, times 0 they are 0."""
    scale = float(torch.tensor(scale, dtype=torch.float32))
    c = form(ctx, k, q_heads, kv_heads, head_dim, scale=scale, seed=42)
    c.q = (c.q.float() * 2.0 ** 59).bfloat16()
    for x in c.keys:
        x[:] = (x.float() * 2.0 ** 59).bfloat16()
    c.write()
    c.device()
    c.check(c.call(), rows=[0, 1, 2, 3, 29, 100, 139])


@pytest.mark.parametrize("form,q_heads,kv_heads,head_dim,ctx,k", FORMS)
@pytest.mark.parametrize("at", [3, 300, 500])
def test_a_value_that_is_not_finite_near_the_newest_keys(form, q_heads, kv_heads, head_dim, ctx, k,
                                                         at):
    """In the newest key but one, which the queries before the last but one do not see: the
    element itself is not finite for those that see it, others of their rows may be; no
    other row, and no other head's, changes."""
    at %= head_dim
    clean = form(ctx, k, q_heads, kv_heads, head_dim, seed=43)
    c = form(ctx, k, q_heads, kv_heads, head_dim, seed=43)
    for b, n in enumerate(ctx):
        c.values[b][n + k - 2, 0, at] = float("inf")
    c.write()
    got = c.device().call().cpu()
    g = q_heads // kv_heads
    for b in {0, len(ctx) - 1}:
        for j in {0, k - 3, k - 2, k - 1} - {-1}:
            want, bound = (x[0] for x in clean.want(b, [j]))
            hit = torch.zeros(q_heads, dtype=torch.bool)
            hit[:g] = j >= k - 2
            assert not got[b, j, hit][:, at].isfinite().any(), (b, j)
            assert ((got[b, j].double() - want).abs() <= bound)[~hit].all(), (b, j)


@pytest.mark.parametrize("form,q_heads,kv_heads,head_dim,ctx,k", FORMS + [
    (base.Case, 10, 2, 512, [200, 900], 40), (base.Case, 5, 1, 256, [30], 60)])
@pytest.mark.parametrize("power", [20, 50, 200])
def test_no_query_changes_anothers_bits(form, q_heads, kv_heads, head_dim, ctx, k, power):
    """Every third query is zero, or of 2^power (200: infinite), or not there (behind its
    request's count): the others' outputs are the same bits."""
    counts = [max(1, k - 1 - b % 3) for b in range(len(ctx))]
    outs = []
    for size in (0.0, 1.0, 2.0 ** power):
        c = form(ctx, k, q_heads, kv_heads, head_dim, counts=counts, seed=44)
        c.q[:, ::3] = (c.q[:, ::3].float() * size).bfloat16()
        for b, n in enumerate(counts):
            c.q[b, n:] = (c.q[b, n:].float() * size).bfloat16()
        outs.append(c.device().call().cpu().view(torch.int16))
    for b, n in enumerate(counts):
        rows = [j for j in range(n) if j % 3]
        for out in outs[1:]:
            assert torch.equal(out[b, rows], outs[0][b, rows]), b
            assert torch.equal(out[b, n:], outs[0][b, n:]), b
