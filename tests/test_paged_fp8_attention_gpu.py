"""Attention over block-scaled e4m3 pages against its definition in 64 bits
(GPU, through the C ABI).  Tolerances: paged_reference.attention_tolerance,
derived from the roundings the kernel makes."""
import math

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Pages in no order, every byte outside a request's keys a NaN, unused
    page-table entries far outside the pool."""

    def __init__(self, key_counts, k, q_heads, kv_heads, head_dim, *, page_rows=128,
                 block_rows=16, window=0, seed=0, scale=None, spread=1.0, pow2=True,
                 scale_spread=3, outliers=False, spare=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.k, self.B = list(key_counts), k, len(key_counts)
        self.hq, self.hkv, self.d = q_heads, kv_heads, head_dim
        self.window = window
        self.scale = 1.0 / math.sqrt(head_dim) if scale is None else scale
        per = max(-(-max(n, 1) // page_rows) for n in key_counts) + spare
        num = sum(-(-max(n, 1) // page_rows) for n in key_counts) + 1
        perm = torch.randperm(num, generator=g).tolist()
        self.table = torch.full((self.B, per), 1 << 30, dtype=torch.int32)
        pool = (num, page_rows, kv_heads, head_dim)
        self.kp = torch.full(pool, 0x7f, dtype=torch.uint8)
        self.vp = torch.full(pool, 0xff, dtype=torch.uint8)
        shape = (num, page_rows // block_rows, kv_heads)

        def scales():
            e = torch.randint(-6 - scale_spread, -6 + scale_spread + 1, shape, generator=g).double()
            if not pow2:
                e = e + torch.rand(shape, generator=g).double()
            return torch.exp2(e).float()

        self.ks, self.vs = scales(), scales()
        self.keys, self.values, self.value_scales = [], [], []
        for b, n in enumerate(self.n):
            pages = [perm.pop() for _ in range(-(-max(n, 1) // page_rows))]
            self.table[b, :len(pages)] = torch.tensor(pages)
            hist = []
            for pool_t, sc in ((self.kp, self.ks), (self.vp, self.vs)):
                x = torch.randn((n, kv_heads, head_dim), generator=g) * 60 * spread
                if outliers:
                    x[torch.rand((n, kv_heads), generator=g) < 0.01] *= 6
                bytes_ = x.clamp(-448, 448).to(ref.E4M3).view(torch.uint8)
                val = ref.decode(bytes_)
                for i, page in enumerate(pages):
                    rows = bytes_[i * page_rows:(i + 1) * page_rows]
                    pool_t[page, :rows.shape[0]] = rows
                    s = sc[page].double().repeat_interleave(block_rows, 0)[:rows.shape[0]]
                    val[i * page_rows:(i + 1) * page_rows] *= s[..., None]
                hist.append(val)
            self.keys.append(hist[0])
            self.values.append(hist[1])
            self.value_scales.append(self.vs[pages].double().repeat_interleave(block_rows, 1)
                                     .flatten(0, 1)[:n])
        self.q = torch.randn((self.B, k, q_heads, head_dim), generator=g).bfloat16()
        self.upload()

    def upload(self):
        self.dev = [x.cuda() for x in (self.q, self.kp, self.vp, self.ks, self.vs, self.table)]
        self.ctx = i32([n - self.k for n in self.n])
        self.ws = carat.workspace_tensor(carat.paged_fp8_workspace_bytes(
            self.B, self.k, self.hq, self.hkv, self.d, self.table.shape[1] * self.kp.shape[1]))
        self.ws.fill_(0xff)

    def call(self, ctx=None, stream=None, out=None, workspace=None, counts=None):
        q, kp, vp, ks, vs, table = self.dev
        if out is None:
            out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
        carat.carat_paged_verify_attention_fp8(
            out, q, kp, vp, ks, vs, table, self.ctx if ctx is None else ctx, scale=self.scale,
            window=self.window, workspace=self.ws if workspace is None else workspace,
            new_counts=counts, stream=stream)
        return out

    def expected(self, b, count=None):
        """Of a request's `count` queries (default all k), the last of which sits
        on its last key."""
        count = self.k if count is None else count
        q = self.q[b, :count].double()
        pos = [self.n[b] - count + j for j in range(count)]
        return ref.attention(q, self.keys[b], self.values[b], pos, self.window, self.scale,
                             self.value_scales[b][:self.n[b]])

    def check(self, out, requests=None):
        out = out.cpu().double()
        for b in range(self.B) if requests is None else requests:
            want, weight = self.expected(b)
            tol = ref.attention_tolerance(want, weight, self.q[b].double(), self.keys[b],
                                          self.scale)
            bad = ~((out[b] - want).abs() <= tol)
            assert not bad.any(), (b, self.n[b], int(bad.sum()),
                                   float(((out[b] - want).abs() / tol).nan_to_num(1e9).max()))

    def run(self):
        out = self.call()
        torch.cuda.synchronize()
        assert carat.carat_get_device_status(clear=True) == 0
        self.check(out)
        return out


CASES = {
    "one_key": dict(key_counts=[1], k=1, q_heads=16, kv_heads=2, head_dim=512),
    "one_key_256": dict(key_counts=[1], k=1, q_heads=2, kv_heads=1, head_dim=256),
    "decode": dict(key_counts=[2, 127, 128, 129, 300, 1500], k=1, q_heads=16, kv_heads=8,
                   head_dim=256, block_rows=32),
    "verify": dict(key_counts=[4, 128, 131, 132, 260, 1000], k=4, q_heads=16, kv_heads=2,
                   head_dim=512, block_rows=64),
    "verify_256": dict(key_counts=[5, 700, 383], k=5, q_heads=8, kv_heads=2, head_dim=256,
                       page_rows=384, block_rows=128),
    "sixteen_rows": dict(key_counts=[16, 500], k=16, q_heads=1, kv_heads=1, head_dim=512),
    "seventeen_rows": dict(key_counts=[40, 513], k=1, q_heads=17, kv_heads=1, head_dim=256),
    "odd_group": dict(key_counts=[33, 900], k=7, q_heads=6, kv_heads=2, head_dim=512),
    "120_rows": dict(key_counts=[15, 640, 129], k=15, q_heads=16, kv_heads=2, head_dim=512),
    "128_rows": dict(key_counts=[16, 400], k=16, q_heads=8, kv_heads=1, head_dim=256),
    "40_rows": dict(key_counts=[20, 1300, 257], k=5, q_heads=16, kv_heads=2, head_dim=512),
    "64_rows_256": dict(key_counts=[16, 900, 5000], k=16, q_heads=8, kv_heads=2, head_dim=256,
                        window=700),
    "80_rows": dict(key_counts=[10, 1100], k=10, q_heads=16, kv_heads=2, head_dim=512),
    "long_120_rows": dict(key_counts=[6000, 2500], k=15, q_heads=16, kv_heads=2, head_dim=512),
    "64_heads": dict(key_counts=[2, 270], k=2, q_heads=64, kv_heads=1, head_dim=512),
    "long": dict(key_counts=[9000], k=2, q_heads=16, kv_heads=2, head_dim=512),
    "long_256": dict(key_counts=[20011], k=1, q_heads=8, kv_heads=4, head_dim=256),
    "outliers": dict(key_counts=[2000, 300], k=4, q_heads=16, kv_heads=2, head_dim=512,
                     outliers=True, spread=0.5),
    "free_scales": dict(key_counts=[700, 90], k=3, q_heads=4, kv_heads=2, head_dim=256,
                        pow2=False),
    "wide_scales": dict(key_counts=[700, 90], k=3, q_heads=4, kv_heads=2, head_dim=512,
                        scale_spread=8, spread=0.2),
    "spare_pages": dict(key_counts=[100, 200], k=2, q_heads=4, kv_heads=4, head_dim=256, spare=5),
    "window": dict(key_counts=[1, 1023, 1024, 1025, 3000], k=1, q_heads=16, kv_heads=8,
                   head_dim=256, window=1024),
    "window_verify": dict(key_counts=[8, 255, 256, 257, 1000], k=8, q_heads=16, kv_heads=2,
                          head_dim=512, window=130, block_rows=32),
    "window_one": dict(key_counts=[4, 500], k=4, q_heads=4, kv_heads=2, head_dim=256, window=1),
    "window_edge": dict(key_counts=[641, 640, 639], k=3, q_heads=4, kv_heads=1, head_dim=512,
                        window=128, page_rows=256, block_rows=128),
    "batch": dict(key_counts=[1 + (i * 97) % 700 for i in range(40)], k=1, q_heads=16, kv_heads=8,
                  head_dim=256),
    "sharp": dict(key_counts=[900, 1300], k=4, q_heads=16, kv_heads=2, head_dim=512, scale=1.0,
                  spread=0.5),
    "negative_scale": dict(key_counts=[300], k=2, q_heads=4, kv_heads=2, head_dim=256,
                           scale=-0.05),
    "zero_scale": dict(key_counts=[300], k=2, q_heads=4, kv_heads=2, head_dim=256, scale=0.0),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_matches_the_definition(name):
    Case(seed=len(name), **CASES[name]).run()


@pytest.mark.parametrize("stale", [0.0, -1.0, float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("shape", [dict(key_counts=[1, 300, 16, 129], k=1, q_heads=16, kv_heads=8,
                                        head_dim=256),
                                   dict(key_counts=[250, 4], k=4, q_heads=16, kv_heads=2,
                                        head_dim=512, block_rows=32)])
def test_scales_of_blocks_without_keys_may_be_anything(shape, stale):
    c = Case(seed=12, **shape)
    R = c.kp.shape[1] // c.ks.shape[1]
    used = torch.zeros(c.ks.shape[:2], dtype=torch.bool)
    for b, n in enumerate(c.n):
        for t in range(0, n, R):
            used[int(c.table[b, t // 128]), t % 128 // R] = True
    c.ks[~used], c.vs[~used] = stale, stale
    c.upload()
    c.run()


@pytest.mark.parametrize("head_dim", [256, 512])
def test_blocks_of_zero_values_keep_their_share(head_dim):
    """Zero values have the least scale, 2^-100: their keys add nothing to the
    sum of values but all of their weight to the denominator."""
    c = Case([700, 130], 3, 8, 2, head_dim, seed=13)
    for b, n in enumerate(c.n):
        for t in range(0, n, 16):
            if t // 16 % 3 == 1:
                page, i = int(c.table[b, t // 128]), t % 128 // 16
                c.vp[page, 16 * i:16 * i + 16] = 0
                c.vs[page, i] = 2.0 ** -100
                c.values[b][t:t + 16] = 0
                c.value_scales[b][t:t + 16] = 2.0 ** -100
    c.upload()
    c.run()


@pytest.mark.parametrize("where", ["key", "value", "key scale", "value scale"])
@pytest.mark.parametrize("q_heads,head_dim,window", [(2, 256, 0), (8, 256, 0), (16, 512, 0),
                                                     (2, 512, 97), (16, 256, 97)])
def test_a_nan_reaches_only_the_queries_that_see_it(where, q_heads, head_dim, window):
    """Request 0's queries sit at 302..305; the NaN is at key 304, the first of its
    block of 16 and seen by the last two, or with a window of 97 at key 207, the last
    of its block, seen by the first two (from 206 and 207 on)."""
    c = Case([306, 200], 4, q_heads, 2, head_dim, seed=14, window=window)
    clean = c.run().clone()
    pos = 207 if window else 304
    page, row = int(c.table[0, pos // 128]), pos % 128
    if where == "key":
        c.kp[page, row, 1, 3] = 0x7f
    elif where == "value":
        c.vp[page, row, 1, head_dim - 3] = 0xff
    else:
        (c.ks if where == "key scale" else c.vs)[page, row // 16, 1] = float("nan")
    c.upload()
    out = c.call()
    torch.cuda.synchronize()
    half = q_heads // 2
    seen = slice(0, 2) if window else slice(2, 4)
    assert out[0, seen, half:].isnan().all()
    out[0, seen, half:] = clean[0, seen, half:]
    assert torch.equal(out.view(torch.int16), clean.view(torch.int16))


RAGGED = {
    "verify": (dict(k=4, q_heads=16, kv_heads=2, head_dim=512), [300, 1, 4, 129, 0, 515],
               [4, 1, 2, 3, 0, 0]),
    "decode": (dict(k=1, q_heads=16, kv_heads=8, head_dim=256), [300, 17, 128], [1, 0, 1]),
    "row_groups": (dict(k=15, q_heads=16, kv_heads=2, head_dim=512), [400, 700, 33, 15],
                   [1, 15, 7, 15]),
    "window": (dict(k=8, q_heads=4, kv_heads=2, head_dim=256, window=50), [400, 55, 1030],
               [5, 8, 1]),
    "long": (dict(k=4, q_heads=16, kv_heads=2, head_dim=512), [30000, 128], [2, 1]),
    "many": (dict(k=4, q_heads=4, kv_heads=2, head_dim=256), [5 + 13 * i % 300 for i in range(400)],
             [i * 7 % 5 for i in range(400)]),
}


@pytest.mark.parametrize("name", sorted(RAGGED))
def test_requests_with_fewer_queries(name):
    """new_counts: the keys end with the last query's (NaN bytes follow), and the
    rows of out behind it stay as they were."""
    shape, key_counts, counts = RAGGED[name]
    c = Case(key_counts, seed=15, **shape)
    ctx = i32([n - m for n, m in zip(key_counts, counts)])
    out = c.call(ctx=ctx, counts=i32(counts)).cpu().double()
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == 0
    for b, m in enumerate(counts):
        assert (out[b, m:] == 3.0).all()
        if m:
            want, weight = c.expected(b, m)
            tol = ref.attention_tolerance(want, weight, c.q[b, :m].double(), c.keys[b], c.scale)
            assert ((out[b, :m] - want).abs() <= tol).all(), b


def test_counts_at_the_capacity_and_out_of_range():
    c = Case([256, 256, 256, 256], 4, 16, 2, 512, seed=16)
    ctx = i32([254, 100, 100, 253])
    out = c.call(ctx=ctx, counts=i32([2, -1, 5, 4]))
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CONTEXT
    assert out[1].isnan().all() and out[2].isnan().all() and out[3].isnan().all()
    want, weight = c.expected(0, 2)
    tol = ref.attention_tolerance(want, weight, c.q[0, :2].double(), c.keys[0], c.scale)
    assert ((out[0, :2].cpu().double() - want).abs() <= tol).all()
    assert (out[0, 2:] == 3.0).all()


def test_several_hundred_requests():
    """More requests than the range search keeps in a warp's first pass, empty and
    rejected ones among them."""
    n = [1 + (i * 37) % 300 for i in range(333)]
    c = Case(n, 1, 2, 1, 256, seed=17)
    ctx, counts = c.ctx.clone(), torch.ones_like(c.ctx)
    ctx[5::50] = -3
    counts[7::50] = 0
    out = c.call(ctx=ctx, counts=counts)
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CONTEXT
    rejected, empty = set(range(5, 333, 50)), set(range(7, 333, 50))
    c.check(out, [b for b in range(333) if b not in rejected | empty])
    assert all(out[b].isnan().all() for b in rejected)
    assert all((out[b] == 3.0).all() for b in empty)


def test_requests_that_share_pages():
    """A common prefix's pages in several requests' tables."""
    c = Case([300, 300, 300], 2, 4, 2, 256, seed=18)
    c.table[1, :2] = c.table[0, :2]
    c.table[2, 0] = c.table[0, 0]
    for x in (c.keys, c.values, c.value_scales):
        x[1][:256] = x[0][:256]
        x[2][:128] = x[0][:128]
    c.upload()
    c.run()


def test_two_graphs_with_one_workspace_on_one_stream():
    a, b = Case([900, 40], 2, 16, 2, 512, seed=19), Case([70, 1500], 2, 16, 2, 512, seed=20)
    need = max(a.ws.numel(), b.ws.numel())
    ws = torch.full((need,), 0xff, dtype=a.ws.dtype, device="cuda")
    outs = [torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda") for c in (a, b)]
    graphs, side = [], torch.cuda.Stream()
    for c, o in zip((a, b), outs):
        c.call(out=o, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            c.call(stream=side, out=o, workspace=ws)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        a.check(outs[0])
        b.check(outs[1])


def test_a_pool_past_32_bits():
    """Pages behind the 2^32-th byte of the pool: bit-equal to the same pages in a
    small pool, through the append and the attention."""
    B, k, hq, hkv, d, R = 2, 4, 16, 8, 512, 32
    rows = (1 << 32) // (hkv * d) + 1024
    num = rows // 128
    g = torch.Generator().manual_seed(23)
    ctx0, ctx = i32([0, 0]), i32([200, 130])
    kn, vn = (torch.randn((B, 200, hkv, d), generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn((B, k, hq, d), generator=g).bfloat16().cuda()
    cs = engine.rotary_table(512, d)
    outs = []
    for pages, first in ((8, 0), (num, num - 8)):
        table = i32([[first + 5, first + 2], [first + 7, first]])
        kp, vp = (torch.empty((pages, 128, hkv, d), dtype=torch.uint8, device="cuda")
                  for _ in range(2))
        ks, vs = (torch.ones((pages, 128 // R, hkv), device="cuda") for _ in range(2))
        carat.carat_paged_rope_append_fp8(kp, vp, ks, vs, table, kn, vn, ctx0, cos_sin=cs,
                                          new_counts=ctx)
        turned = torch.empty_like(q)
        carat.carat_paged_rope_append_fp8(kp, vp, ks, vs, table, kn[:, :k].contiguous(),
                                          vn[:, :k].contiguous(), ctx, cos_sin=cs, queries=q,
                                          queries_out=turned)
        ws = carat.workspace_tensor(carat.paged_fp8_workspace_bytes(B, k, hq, hkv, d, 256))
        out = torch.zeros_like(q)
        carat.carat_paged_verify_attention_fp8(out, turned, kp, vp, ks, vs, table, ctx, scale=0.05,
                                               workspace=ws)
        got = [out.view(torch.int16), turned.view(torch.int16)]
        for x in (kp, vp):
            for b, n in enumerate((204, 134)):
                got.append(x[table[b].long()].flatten(0, 1)[:n].clone())
        outs.append(got)
        del kp, vp
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == 0
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    assert outs[0][0].view(torch.bfloat16).isfinite().all()


def test_steps_in_a_row_without_waiting():
    """Appends and attentions follow each other on one stream, each starting while
    the one before drains: the same bits as with a wait after every call."""
    B, k, hq, hkv, d = 5, 4, 16, 2, 512
    g = torch.Generator().manual_seed(22)
    cs = engine.rotary_table(1024, d)
    steps = [[torch.randn((B, k, h, d), generator=g).bfloat16().cuda() for h in (hq, hkv, hkv)]
             for _ in range(40)]
    ctxs = [i32([50 * b + 3 * i for b in range(B)]) for i in range(40)]
    results = []
    for wait in (True, False):
        pool = engine.SharedPool(num_pages=16, page_bytes=128 * hkv * d * 2, pages_per_ring=4,
                                 fill=0.0)
        table = i32([pool.alloc.alloc_pages(3) for _ in range(B)])
        layer = engine.Fp8PagedLayer(pool, table, cs, q_heads=hq, kv_heads=hkv, head_dim=d,
                                     max_proposals=k)
        first = torch.randn((B, 256, hkv, d), generator=torch.Generator().manual_seed(1))
        layer.append(first.bfloat16().cuda(), first.bfloat16().cuda(), i32([0] * B),
                     new_counts=ctxs[0])
        torch.cuda.synchronize()
        outs = []
        for (q, kn, vn), ctx in zip(steps, ctxs):
            outs.append(layer.step(q, kn, vn, ctx))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append(torch.stack(outs))
    assert torch.equal(results[0].view(torch.int16), results[1].view(torch.int16))
    assert results[0].isfinite().all()


def test_small_weights_of_a_long_tail_survive():
    """One key holds half the mass and 8191 share the rest: each weight is
    2^-13 of the largest, and their sum must not be lost."""
    c = Case([8192], 1, 2, 1, 256, seed=2, scale=1.0)
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.kp[:, :, 0, :] = 0
    page, row = int(c.table[0, 3]), 5
    t = 3 * 128 + row
    c.ks.fill_(2.0 ** -4)
    one = torch.tensor(9.0).to(ref.E4M3).view(torch.uint8)     # score 16 * 9 / 16 = 9
    c.q[..., 0] = 16.0
    c.kp[page, row, 0, 0] = one
    c.keys[0].zero_()
    c.keys[0][t, 0, 0] = 9.0 / 16.0
    c.upload()
    want, _ = c.expected(0)
    out = c.call().cpu().double()
    c.check(out)
    share = math.exp(9.0) / (math.exp(9.0) + 8191)
    assert 0.4 < share < 0.6
    lone = share * c.values[0][t, 0]
    assert (want - lone).abs().max() > 1e-3      # the tail is visible at all


@pytest.mark.parametrize("row_spread", [1e-3, 1e3])
def test_rows_of_very_different_size(row_spread):
    """Query rows of one unit whose magnitudes differ by powers of ten keep
    their own precision."""
    c = Case([400, 90], 4, 8, 1, 256, seed=3)
    f = torch.ones(1, 4, 8, 1)
    f[:, 1::2] = row_spread
    f[:, :, ::2] /= row_spread ** 0.5
    c.q = (c.q * f).bfloat16()
    c.scale = 1e-3
    c.upload()
    c.run()


def test_non_finite_queries_stay_in_their_rows():
    c = Case([300, 50], 4, 8, 2, 512, seed=4)
    clean = c.run().clone()
    c.q[0, 1, 3, 7] = float("nan")
    c.q[1, 2, 0, 100] = float("inf")
    c.upload()
    out = c.call()
    assert out[0, 1, 3].isnan().all() and out[1, 2, 0].isnan().all()
    out[0, 1, 3] = clean[0, 1, 3]
    out[1, 2, 0] = clean[1, 2, 0]
    assert torch.equal(out.view(torch.int16), clean.view(torch.int16))


def test_zero_queries_and_subnormal_queries():
    c = Case([200], 3, 4, 2, 256, seed=5)
    c.q[0, 0] = 0.0
    c.q[0, 1] = (c.q[0, 1].float() * 2.0 ** -127).bfloat16()
    c.upload()
    c.run()


def test_rejected_requests_among_valid_ones():
    c = Case([100, 200, 300, 400], 4, 16, 2, 512, seed=6)
    ref_out = c.run().clone()
    cap = c.table.shape[1] * 128
    ctx = c.ctx.clone()
    ctx[1], ctx[3] = -1, cap - 3
    out = c.call(ctx=ctx)
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CONTEXT
    assert out[1].isnan().all() and out[3].isnan().all()
    for b in (0, 2):
        c.check(out, [b])


def test_a_page_outside_the_pool_reads_as_zeros():
    """Its keys score 0 and its values are 0; the status says so."""
    c = Case([300, 100], 2, 4, 2, 256, seed=7)
    c.table[0, 1] = -7
    c.keys[0][128:256] = 0
    c.values[0][128:256] = 0
    c.upload()
    out = c.call()
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CACHE_ID
    c.check(out)


def test_repeated_calls_give_identical_bits():
    c = Case([5000, 700, 30, 2200], 4, 16, 2, 512, seed=8)
    first = c.run()
    for _ in range(20):
        assert torch.equal(c.call().view(torch.int16), first.view(torch.int16))


def test_two_streams_with_two_workspaces():
    c = Case([3000, 400], 2, 16, 2, 512, seed=9)
    first = c.run()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [c.ws, torch.full_like(c.ws, 0x55)]
    outs = [[torch.zeros_like(first) for _ in range(8)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(8):
        for s, ws, o in zip(streams, spaces, outs):
            c.call(stream=s, out=o[i], workspace=ws)
    torch.cuda.synchronize()
    for o in outs:
        for x in o:
            assert torch.equal(x.view(torch.int16), first.view(torch.int16))


def test_captured_calls_read_the_lengths_at_replay():
    c = Case([700, 900], 2, 8, 2, 256, seed=10)
    out = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    full = c.run().clone()
    ctx = c.ctx.clone()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        c.call(ctx=ctx, stream=side, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), full.view(torch.int16))
    ctx.copy_(i32([98, 3]))
    graph.replay()
    torch.cuda.synchronize()
    c.n = [100, 5]
    c.check(out)


def test_refusals():
    c = Case([100, 90], 2, 4, 2, 256, seed=11)
    q, kp, vp, ks, vs, table = c.dev
    out = torch.zeros_like(q)

    def refused(error, **kw):
        a = dict(out=out, q=q, kp=kp, vp=vp, ks=ks, vs=vs, table=table, ctx=c.ctx, ws=c.ws,
                 window=0, scale=0.1, counts=None)
        a.update(kw)
        with pytest.raises(error) as e:
            carat.carat_paged_verify_attention_fp8(
                a["out"], a["q"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["ctx"],
                scale=a["scale"], window=a["window"], workspace=a["ws"],
                new_counts=a["counts"])
        return e.value

    refused(TypeError, out=out.float())
    refused(TypeError, q=q.half())
    refused(TypeError, kp=kp.view(torch.int8))
    refused(ValueError, vp=vp[1:])
    refused(ValueError, kp=kp[..., :128].contiguous(), vp=vp[..., :128].contiguous())
    refused(ValueError, ks=ks[:, :, :1], vs=vs[:, :, :1])
    refused(ValueError, ks=ks[1:], vs=vs[1:])
    refused(ValueError, table=table[:1])
    refused(ValueError, table=table.cpu())
    refused(ValueError, ctx=c.ctx[:1])
    refused(ValueError, out=out[:1])
    refused(ValueError, q=q.transpose(1, 2).contiguous().transpose(1, 2))
    refused(TypeError, counts=torch.ones_like(c.ctx).long())
    refused(ValueError, counts=torch.ones_like(c.ctx)[:1])
    refused(ValueError, counts=torch.ones_like(c.ctx).cpu())
    assert refused(carat.CaratError, window=-1).status == carat.CARAT_ERR_INVALID_ARG
    assert refused(carat.CaratError, scale=float("nan")).status == carat.CARAT_ERR_INVALID_ARG
    assert refused(carat.CaratError, ws=c.ws[:16]).status == carat.CARAT_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == 0


def test_layer_steps_match_the_definition():
    """Prompt, then verify steps through Fp8PagedLayer in a DecodeStep: the
    cache's contents are read back after each step, and the output must be the
    attention of the rotated queries over exactly those."""
    B, k, hq, hkv, d = 3, 4, 16, 2, 512
    page_bytes = 128 * hkv * d
    pool = engine.SharedPool(num_pages=24, page_bytes=page_bytes, pages_per_ring=4,
                             fill=float("nan"))
    table = torch.tensor([pool.alloc.alloc_pages(4) for _ in range(B)], dtype=torch.int32)
    cs = engine.rotary_table(4 * 128, d, base=1e6)
    g = torch.Generator().manual_seed(21)

    def rows(n, h):
        return torch.randn((B, n, h, d), generator=g).bfloat16().cuda()

    for window in (0, 200):
        layer = engine.Fp8PagedLayer(pool, table.cuda(), cs, q_heads=hq, kv_heads=hkv, head_dim=d,
                                     max_proposals=k, block_rows=32, window=window)
        counts = [300, 1, 129]
        layer.append(rows(300, hkv), rows(300, hkv), i32([0] * B), new_counts=i32(counts))
        ctx = i32(counts)
        q, kn, vn = rows(k, hq), rows(k, hkv), rows(k, hkv)
        step = engine.DecodeStep([layer], [(q, kn, vn, ctx)])
        assert step.outputs[0].dtype == torch.bfloat16
        have = list(counts)
        for it in range(4):
            q.copy_(rows(k, hq)), kn.copy_(rows(k, hkv)), vn.copy_(rows(k, hkv))
            ctx.copy_(i32(have))
            if it == 2:
                step.capture()       # runs the step once more on the same rows
                step.replay()
            elif it == 3:
                step.replay()
            else:
                step.run()
            torch.cuda.synchronize()
            out = step.outputs[0].cpu().double()
            kp, vp = layer.key_pages.cpu(), layer.value_pages.cpu()
            for b in range(B):
                n = have[b] + k
                pages = table[b].long()
                keys, values = (
                    (ref.decode(p)[pages] * s.cpu().double()[pages].repeat_interleave(32, 1)[
                        ..., None]).flatten(0, 1)[:n]
                    for p, s in ((kp, layer.k_scales), (vp, layer.v_scales)))
                pos = [have[b] + j for j in range(k)]
                turned = torch.stack([ref.rotate(q[b, j].cpu().double(), cs.cpu(), pos[j], False)
                                      for j in range(k)])
                want, weight = ref.attention(turned, keys, values, pos, window, layer.scale)
                # the rotated queries are rounded to bf16: a relative 2^-8 of each
                # product moves a score by at most 2^-8 sum |q k|
                a = ref.score_magnitude(turned, keys, layer.scale)
                tol = ref.attention_tolerance(want, weight, turned, keys, layer.scale) \
                    + 2 * math.expm1(2.0 ** -8 * a) * weight
                assert ((out[b] - want).abs() <= tol).all(), (window, it, b)
                have[b] += 1 + b          # some proposals are rejected
    assert carat.carat_get_device_status(clear=True) == 0


def test_bf16_pages_after_the_rotary_append():
    """PagedGlobalLayer with a rotary table: step() equals rotating on the host
    and taking the fused unrotated step, up to the rounding of its inputs."""
    B, k, hq, hkv, d = 3, 4, 16, 2, 512
    page_bytes = 256 * hkv * d
    pool = engine.SharedPool(num_pages=16, page_bytes=page_bytes, pages_per_ring=4, fill=0.0)
    cs = engine.rotary_table(512, d, base=1e6)
    table = torch.tensor([pool.alloc.alloc_pages(4) for _ in range(B)], dtype=torch.int32).cuda()
    layer = engine.PagedGlobalLayer(pool, table, q_heads=hq, kv_heads=hkv, head_dim=d,
                                    max_proposals=k, cos_sin=cs)
    g = torch.Generator().manual_seed(22)

    def rows(n, h):
        return torch.randn((B, n, h, d), generator=g).bfloat16().cuda()

    counts = [300, 2, 130]
    layer.append(rows(300, hkv), rows(300, hkv), i32([0] * B), new_counts=i32(counts))
    q, kn, vn, ctx = rows(k, hq), rows(k, hkv), rows(k, hkv), i32(counts)
    out = layer.step(q, kn, vn, ctx).cpu().double()
    for b in range(B):
        n = counts[b] + k
        keys, values = (p.cpu()[table[b].long().cpu()].flatten(0, 1)[:n].double()
                        for p in (layer.key_pages, layer.value_pages))
        turned = layer.rotated.view(B, k, hq, d)[b].cpu().double()
        pos = [counts[b] + j for j in range(k)]
        want, weight = ref.attention(turned, keys, values, pos, 0, layer.scale)
        # weights rounded to bf16 (2^-8), scores accumulated in fp32
        a = ref.score_magnitude(turned, keys, layer.scale)
        tol = 2 * (2.0 ** -8 + a * (d + 64) * 2.0 ** -24) * weight + 2.0 ** -20 * want.abs()
        assert ((out[b] - want).abs() <= tol).all(), b
        for j in range(k):
            x = q[b, j].cpu().double()
            y = ref.rotate(x, cs.cpu(), pos[j], False)
            t = 2.0 ** -8 * y.abs() + 2.0 ** -22 * ref.pair_magnitude(x, cs.cpu(), False)
            assert ((turned[j] - y).abs() <= t).all()
    assert carat.carat_get_device_status(clear=True) == 0


@pytest.mark.parametrize("window", [0, 150])
def test_ragged_layer_steps_over_stale_memory(window):
    """step() with counts per request, over pages and scales that hold NaNs
    wherever nothing was appended: rows within a count match the definition,
    rows behind it stay as they were."""
    B, k, hq, hkv, d, R = 4, 4, 16, 2, 512, 16
    pool = engine.SharedPool(num_pages=16, page_bytes=128 * hkv * d, pages_per_ring=4,
                             fill=float("nan"))
    table = torch.tensor([pool.alloc.alloc_pages(3) for _ in range(B)], dtype=torch.int32)
    cs = engine.rotary_table(384, d)
    layer = engine.Fp8PagedLayer(pool, table.cuda(), cs, q_heads=hq, kv_heads=hkv, head_dim=d,
                                 max_proposals=k, block_rows=R, window=window)
    layer.k_scales.fill_(float("nan"))
    layer.v_scales.fill_(float("nan"))
    g = torch.Generator().manual_seed(41)

    def rows(n, h):
        return torch.randn((B, n, h, d), generator=g).bfloat16().cuda()

    have = [207, 127, 1, 32]
    layer.append(rows(207, hkv), rows(207, hkv), i32([0] * B), new_counts=i32(have))
    for counts in ([4, 2, 1, 0], [1, 0, 4, 3]):
        q = rows(k, hq)
        out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
        layer.step(q, rows(k, hkv), rows(k, hkv), i32(have), out=out, new_counts=i32(counts))
        torch.cuda.synchronize()
        out = out.cpu().double()
        for b, m in enumerate(counts):
            assert (out[b, m:] == 3.0).all()
            if not m:
                continue
            n, pages = have[b] + m, table[b].long()
            keys, values = (
                (ref.decode(p.cpu())[pages]
                 * s.cpu().double()[pages].repeat_interleave(R, 1)[..., None]).flatten(0, 1)[:n]
                for p, s in ((layer.key_pages, layer.k_scales), (layer.value_pages, layer.v_scales)))
            pos = [have[b] + j for j in range(m)]
            turned = torch.stack([ref.rotate(q[b, j].cpu().double(), cs.cpu(), pos[j], False)
                                  for j in range(m)])
            want, weight = ref.attention(turned, keys, values, pos, window, layer.scale)
            # the rotated queries are rounded to bf16, as in the test above
            a = ref.score_magnitude(turned, keys, layer.scale)
            tol = ref.attention_tolerance(want, weight, turned, keys, layer.scale) \
                + 2 * math.expm1(2.0 ** -8 * a) * weight
            assert ((out[b, :m] - want).abs() <= tol).all(), (counts, b)
        have = [n + m for n, m in zip(have, counts)]
    assert carat.carat_get_device_status(clear=True) == 0


def test_different_calls_at_once():
    """Three shapes of tile on three streams at the same time, each with its own
    workspace: the same bits as one after the other."""
    cases = [Case([3000, 700, 90, 1500], 1, 16, 8, 256, seed=50, window=1024),
             Case([2500, 300], 4, 16, 2, 512, seed=51),
             Case([1800, 640], 15, 16, 2, 512, seed=52)]
    first = [c.run().clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.zeros_like(f) for _ in range(30)] for f in first]
    torch.cuda.synchronize()
    for i in range(30):
        for c, s, o in zip(cases, streams, outs):
            c.call(stream=s, out=o[i])
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == 0
    for f, o in zip(first, outs):
        for x in o:
            assert torch.equal(x.view(torch.int16), f.view(torch.int16))
