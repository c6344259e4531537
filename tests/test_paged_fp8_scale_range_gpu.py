"""Attention over e4m3 pages at the ends of the value scales' range, 2^-100 to
2^100: the softmax's denominator does not depend on the value scales, however
far they lie apart and whatever order they come in (GPU, against 64 bits;
tolerances: paged_reference.attention_tolerance)."""
import math

import pytest
import torch

import paged_reference as ref
from sliding_window_gqa_ring_gb300 import carat
from test_paged_fp8_attention_gpu import Case

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -100


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    carat.library()
    carat.carat_get_device_status(clear=True)
    yield
    assert carat.carat_get_device_status(clear=True) == 0


def set_value_scales(c, b, scale_of_tile):
    """Gives the 128-key tiles of request b the value scales scale_of_tile(i), on
    the same bytes, or all-zero bytes under the least scale where it says None."""
    rows = c.kp.shape[1]
    per = rows // c.vs.shape[1]
    for i in range(-(-c.n[b] // 128)):
        scale = scale_of_tile(i)
        page, r0 = int(c.table[b, 128 * i // rows]), 128 * i % rows
        if scale is None:
            c.vp[page, r0:r0 + 128][:max(0, c.n[b] - 128 * i)] = 0
        c.vs[page, r0 // per:(r0 + 128) // per] = TINY if scale is None else scale
        held = slice(128 * i, min(128 * i + 128, c.n[b]))
        bytes_ = c.vp[page, r0:r0 + held.stop - held.start]
        c.values[b][held] = ref.decode(bytes_) * (TINY if scale is None else scale)
        c.value_scales[b][held] = TINY if scale is None else scale


def repeat(c, batch, seed):
    """The case's one request `batch` times over, on the same pages, with queries
    of their own: enough units that a CTA walks whole ones."""
    c.n, c.B, c.table = c.n * batch, batch, c.table.repeat(batch, 1)
    c.keys, c.values, c.value_scales = c.keys * batch, c.values * batch, c.value_scales * batch
    c.q = torch.randn((batch, *c.q.shape[1:]), generator=torch.Generator().manual_seed(seed)
                      ).bfloat16()


ORDERS = {
    "zeros first": lambda n, big: lambda i: None if i < n // 2 else big,
    "zeros last": lambda n, big: lambda i: big if i < n // 2 else None,
    "in turn": lambda n, big: lambda i: None if i % 2 == 0 else big,
    "rising": lambda n, big: lambda i: (None, 2.0 ** -40, 1.0, big)[min(3, 4 * i // n)],
}
SHAPES = {
    "8 rows": dict(k=1, q_heads=8, kv_heads=1, head_dim=256),
    "16 rows": dict(k=4, q_heads=4, kv_heads=1, head_dim=256),
    "32 rows": dict(k=4, q_heads=16, kv_heads=2, head_dim=512, block_rows=64),
    "40 rows": dict(k=5, q_heads=8, kv_heads=1, head_dim=512),
}


@pytest.mark.parametrize("order", sorted(ORDERS))
@pytest.mark.parametrize("exponent", [0, 27, 30, 100])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_whole_tiles_of_zero_values_keep_their_share_over_pieces(shape, exponent, order):
    """Few requests: a tile or two of a unit to a CTA, joined by the merge."""
    c = Case([1500, 700], seed=61, **SHAPES[shape])
    for b, n in enumerate(c.n):
        set_value_scales(c, b, ORDERS[order](-(-n // 128), 2.0 ** exponent))
    c.upload()
    c.run()


@pytest.mark.parametrize("order", sorted(ORDERS))
@pytest.mark.parametrize("exponent", [0, 30, 100])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_whole_tiles_of_zero_values_keep_their_share_within_a_cta(shape, exponent, order):
    """Many requests on the same pages: the running sum is rescaled from tile to
    tile."""
    c = Case([1000], seed=62, **SHAPES[shape])
    set_value_scales(c, 0, ORDERS[order](8, 2.0 ** exponent))
    repeat(c, 330, seed=63)
    c.upload()
    out = c.call()
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == 0
    c.check(out, range(0, 330, 11))


@pytest.mark.parametrize("q_heads,k", [(8, 1), (8, 2)])
def test_a_long_sum_under_the_least_scale(q_heads, k):
    """40000 keys of scale 2^-100 whose scores lie 7.75 octaves above the first
    tile's: the sum of 2^(score - maximum) is 2^129.5 where the maximum is that of
    the weighted scores and has not moved."""
    n = 40000
    c = Case([n], k, q_heads, 1, 256, seed=64, scale=7.75 * math.log(2.0), spread=0.5)
    g = torch.Generator().manual_seed(65)
    x = (torch.rand((n, 1, 256), generator=g) * 100 + 20).to(ref.E4M3).view(torch.uint8)
    c.ks.fill_(1.0), c.vs.fill_(TINY)
    for i in range(-(-n // 128)):
        page, m = int(c.table[0, i]), min(128, n - 128 * i)
        c.kp[page, :m] = 0
        if i > 0:
            c.kp[page, :m, 0, 0] = 0x38                                # 1.0
        c.vp[page, :m] = x[128 * i:128 * i + m]
    c.keys[0].zero_()
    c.keys[0][128:, 0, 0] = 1.0
    c.values[0] = ref.decode(x) * TINY
    c.value_scales[0].fill_(TINY)
    c.q.zero_()
    c.q[..., 0] = 1.0
    one = c.q
    repeat(c, 304, seed=66)
    c.q = one.repeat(304, 1, 1, 1)
    c.upload()
    out = c.call()
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == 0
    c.check(out, [0])
    want = out[:1].view(torch.int16)
    # (units that are cut add up in another order)
    whole = (out.view(torch.int16) == want).flatten(1).all(1)
    assert whole.sum() >= 152
    assert ((out.float() / out[:1].float() - 1).abs() <= 2.0 ** -7).all()


@pytest.mark.parametrize("kw", [dict(k=1, q_heads=8, kv_heads=1, head_dim=256),
                                dict(k=4, q_heads=16, kv_heads=2, head_dim=512),
                                dict(k=3, q_heads=4, kv_heads=1, head_dim=256, window=200)])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("distinct", [False, True])
@pytest.mark.parametrize("batch", [1, 330])
def test_scores_of_keys_under_the_largest_scale(kw, sign, distinct, batch):
    """Key scales of 2^100: scores of +-3e31 in log2 units, all alike, or every
    seventh key's half of that (then the smaller magnitude, or the larger value, takes
    all)."""
    c = Case([700], seed=67, scale=1.0 / 16.0, **kw)
    c.ks.fill_(2.0 ** 100)
    c.q.zero_()
    c.q[..., 0] = 16.0
    c.keys[0].zero_()
    for t in range(700):
        half = distinct and t % 7 == 3
        page, row = int(c.table[0, t // 128]), t % 128
        c.kp[page, row] = 0
        c.kp[page, row, :, 0] = (0x80 if sign < 0 else 0) | (0x50 if half else 0x58)   # 8, 16
        c.keys[0][t, :, 0] = sign * (8.0 if half else 16.0) * 2.0 ** 100
    if batch > 1:
        q = c.q
        repeat(c, batch, seed=68)
        c.q = q.repeat(batch, 1, 1, 1)
    c.upload()
    out = c.call()
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == 0
    for b in {0, batch - 1, batch // 2}:
        want, weight = c.expected(b)
        # (the scores are exact: powers of two and equal products)
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -10 * (1 + 2.0 ** -8) * weight
        assert ((out[b].cpu().double() - want).abs() <= tol).all(), b


@pytest.mark.parametrize("exponent", [-93, -100, -110, -118])
@pytest.mark.parametrize("kw", [dict(k=2, q_heads=8, kv_heads=1, head_dim=256),
                                dict(k=4, q_heads=16, kv_heads=2, head_dim=512)])
def test_small_queries_meet_large_key_scales(kw, exponent):
    """Queries of 2^-118 to 2^-93 and key scales that make ordinary scores of them
    keep the precision of ordinary queries."""
    c = Case([500, 130], seed=69, scale=2.0 ** (-exponent - 100 - 10), **kw)
    c.ks.fill_(2.0 ** 100)
    for b, n in enumerate(c.n):
        for i in range(-(-n // 128)):
            m = min(128, n - 128 * i)
            c.keys[b][128 * i:128 * i + m] = ref.decode(c.kp[int(c.table[b, i]), :m]) * 2.0 ** 100
    c.q = (c.q.double() * 2.0 ** exponent).bfloat16()
    c.upload()
    c.run()
