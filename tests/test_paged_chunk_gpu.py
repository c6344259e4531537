"""Attention of a chunk of new tokens over bf16 pages against its definition in 64 bits
(GPU, through the C ABI).  Tolerance: tests/chunk_reference.py."""
import math

import pytest
import torch

import chunk_reference as ref
from sliding_window_gqa_ring_gb300 import carat

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    carat.library()
    carat.carat_get_device_status(clear=True)
    yield
    assert carat.carat_get_device_status(clear=True) == 0


class Case:
    """Pages with known contents under a table in no order; every row that holds no key of
    its request, every page of nobody and every row of `out` behind a count holds NaNs."""

    def __init__(self, ctx, k, q_heads, kv_heads, head_dim, *, page_rows=128, counts=None,
                 window=0, sinks=0, seed=0, spread=1.0, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.k, self.B = list(ctx), k, len(ctx)
        self.counts = list(counts) if counts is not None else None
        self.n = self.counts or [k] * self.B
        self.window, self.sinks, self.page_rows = window, sinks, page_rows
        self.scale = 1.0 / math.sqrt(head_dim) if scale is None else scale
        per = max(1, -(-max(max(c, 0) + k for c in ctx) // page_rows))
        self.num_pages = self.B * per + 3
        self.table = torch.randperm(self.num_pages, generator=g)[:self.B * per].view(
            self.B, per).to(torch.int32)
        pool = (self.num_pages, page_rows, kv_heads, head_dim)
        self.kp = torch.full(pool, float("nan"), dtype=torch.bfloat16)
        self.vp = torch.full(pool, float("nan"), dtype=torch.bfloat16)
        self.keys, self.values = [], []
        for b in range(self.B):
            m = max(self.ctx[b], 0) + max(0, min(self.n[b], k))
            kk = torch.randn((m, kv_heads, head_dim), generator=g).bfloat16()
            vv = torch.randn((m, kv_heads, head_dim), generator=g).bfloat16()
            self.keys.append(kk)
            self.values.append(vv)
        self.write()
        self.q = (torch.randn((self.B, k, q_heads, head_dim), generator=g) * spread).bfloat16()

    def write(self):
        for b in range(self.B):
            for x, pages in ((self.keys[b], self.kp), (self.values[b], self.vp)):
                for i in range(0, x.shape[0], self.page_rows):
                    part = x[i:i + self.page_rows]
                    pages[self.table[b, i // self.page_rows], :part.shape[0]] = part

    def device(self):
        self.dq, self.dk, self.dv = self.q.cuda(), self.kp.cuda(), self.vp.cuda()
        self.dt = self.table.cuda()
        self.dc = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        self.dn = (torch.tensor(self.counts, dtype=torch.int32, device="cuda")
                   if self.counts is not None else None)
        self.out = torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        B, k, hq, d = self.q.shape
        need = carat.paged_chunk_workspace_bytes(B, k, hq, self.kp.shape[2], d)
        # a workspace that holds NaNs: it needs no initialisation
        self.ws = carat.workspace_tensor(need).fill_(0xff) if need else None
        return self

    def call(self, **kw):
        carat.carat_paged_chunk_attention(
            self.out, self.dq, self.dk, self.dv, self.dt, self.dc, scale=self.scale,
            window=self.window, sinks=self.sinks, new_counts=self.dn, workspace=self.ws, **kw)
        return self.out

    def want(self, b, rows=None):
        rows = range(self.n[b]) if rows is None else rows
        if not len(rows):
            return None
        parts = [ref.attention(self.q[b, j:j + 1].double(), self.keys[b].double(),
                               self.values[b].double(), self.ctx[b] + j, self.window, self.sinks,
                               self.scale) for j in rows]
        return tuple(torch.cat(x) for x in zip(*parts))

    def check(self, out, rows=None):
        out = out.cpu()
        for b in range(self.B):
            r = list(range(self.n[b])) if rows is None else [j for j in rows if j < self.n[b]]
            if r:
                want, bound = self.want(b, r)
                got = out[b, r].double()
                assert got.isfinite().all(), (b, "not finite")
                off = (got - want).abs() - bound
                assert (off <= 0).all(), (b, float(off.max()), off.argmax())
            assert (out[b, self.n[b]:] == 7.0).all(), (b, "rows behind the count")


SHAPES = [(16, 2, 512), (16, 8, 256), (3, 1, 256), (5, 1, 512), (4, 4, 256), (64, 1, 256)]


@pytest.mark.parametrize("q_heads,kv_heads,head_dim", SHAPES)
@pytest.mark.parametrize("k,ctx", [
    (1, [0]), (1, [1, 126, 127, 128, 1000]), (4, [0, 125, 700]), (17, [0, 111, 112, 113]),
    (64, [64, 300]), (129, [0, 127]), (300, [5])])
def test_lengths(k, ctx, q_heads, kv_heads, head_dim):
    c = Case(ctx, k, q_heads, kv_heads, head_dim, seed=k, spread=2.0).device()
    c.check(c.call())


@pytest.mark.parametrize("q_heads,kv_heads,head_dim", [(16, 2, 512), (16, 8, 256), (6, 2, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 5), (127, 4), (128, 0), (129, 128),
                                          (200, 130), (300, 1), (1 << 30, 3), (50, 1 << 30)])
@pytest.mark.parametrize("k,ctx", [(1, [0, 40, 900]), (3, [129, 640]), (200, [0, 333])])
def test_windows_and_sinks(window, sinks, k, ctx, q_heads, kv_heads, head_dim):
    c = Case(ctx, k, q_heads, kv_heads, head_dim, window=window, sinks=sinks, seed=window,
             page_rows=256, spread=2.0).device()
    c.check(c.call())


@pytest.mark.parametrize("q_heads,kv_heads,head_dim", [(16, 2, 512), (8, 4, 256)])
@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("counts,ctx,k", [([5, 0, 1, 40], [0, 70, 300, 127], 40),
                                          ([0, 0], [3, 4], 5), ([130, 257, 0, 1], [1, 0, 0, 0], 257)])
def test_counts(counts, ctx, k, window, q_heads, kv_heads, head_dim):
    c = Case(ctx, k, q_heads, kv_heads, head_dim, counts=counts, window=window, sinks=2,
             seed=7).device()
    c.check(c.call())


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,window,sinks", [
    (16, 2, 512, 0, 0), (16, 8, 256, 1024, 4), (2, 1, 512, 700, 300), (16, 8, 256, 0, 0)])
def test_long_contexts(q_heads, kv_heads, head_dim, window, sinks):
    c = Case([9000, 20000], 3, q_heads, kv_heads, head_dim, window=window, sinks=sinks, seed=3,
             spread=3.0, page_rows=384).device()
    c.check(c.call())


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,window", [(16, 2, 512, 0), (16, 8, 256, 1024)])
def test_a_long_chunk(q_heads, kv_heads, head_dim, window):
    c = Case([500], 2500, q_heads, kv_heads, head_dim, window=window, sinks=100, seed=4,
             spread=2.0).device()
    out = c.call()
    c.check(out, rows=[0, 1, 17, 127, 128, 600, 1023, 1024, 1600, 2047, 2400, 2498, 2499])


@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-30, 3.0, 1e4])
@pytest.mark.parametrize("head_dim", [256, 512])
def test_scales(scale, head_dim):
    """Flat, inverted and one-hot softmaxes.  (At 1e4 the scores' fp32 rounding alone moves
    every weight, so there the one-hot result is compared where it is one.)"""
    c = Case([200], 30, 4, 2, head_dim, scale=scale, seed=5).device()
    out = c.call()
    if abs(scale) < 1:
        c.check(out)
        return
    got = out.cpu()[0].double()
    assert got.isfinite().all()
    for j in range(30):
        for h in range(4):
            s = (c.q[0, j, h].double() @ c.keys[0][:200 + j + 1, h // 2].double().T) * scale
            top = s.topk(2).values
            if top[0] - top[1] > 40 + abs(scale) * 1e-2:
                want = c.values[0][int(s.argmax()), h // 2].double()
                assert ((got[j, h] - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -20).all()


def test_rising_scores_move_the_running_maximum():
    """Keys whose scores grow from tile to tile, by far more than any slack, and back."""
    for head_dim in (256, 512):
        c = Case([700], 60, 4, 2, head_dim, seed=6)
        direction = torch.ones(head_dim)
        c.q[:] = direction.bfloat16() * 0.5
        for x, sign in ((c.keys[0], 1.0),):
            n = x.shape[0]
            ramp = torch.cat([torch.linspace(-4, 4, n // 2), torch.linspace(4, -4, n - n // 2)])
            x[:] = (x.float() * 0.05 + sign * ramp[:, None, None]).bfloat16()
        c.write()
        c.device()
        c.check(c.call())


@pytest.mark.parametrize("head_dim", [256, 512])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_reach_only_the_queries_that_see_them(bad, head_dim):
    """In key 290 (value and key rows): queries before it and, under the window, long after
    it are as without."""
    for where in ("v", "k"):
        for window in (0, 40):
            clean = Case([250], 120, 4, 2, head_dim, window=window, sinks=3, seed=8)
            c = Case([250], 120, 4, 2, head_dim, window=window, sinks=3, seed=8)
            rows = c.values[0] if where == "v" else c.keys[0]
            rows[290, 1, 5] = bad
            c.write()
            got = c.device().call().cpu()[0]
            want, bound = clean.want(0)
            for j in range(120):
                sees = bool(ref.seen(250 + j, 370, window, 3)[290])
                for h in range(4):
                    if sees and h // 2 == 1:
                        if where == "v":
                            assert not got[j, h, 5].isfinite(), (j, h)
                    else:
                        assert ((got[j, h].double() - want[j, h]).abs() <= bound[j, h]).all(), (j, h)


@pytest.mark.parametrize("head_dim", [256, 512])
def test_a_non_finite_value_that_every_query_sees_stays_in_its_element(head_dim):
    c = Case([2000], 5, 4, 2, head_dim, seed=9)
    c.values[0][100, 0, 7] = float("inf")
    c.write()
    clean = Case([2000], 5, 4, 2, head_dim, seed=9)
    want, bound = clean.want(0)
    got = c.device().call().cpu()[0].double()
    assert not got[:, :2, 7].isfinite().any()
    ok = torch.ones_like(got, dtype=torch.bool)
    ok[:, :2, 7] = False
    assert ((got - want).abs() <= bound)[ok].all()


def test_queries_that_are_not_finite_stay_in_their_rows():
    for head_dim in (256, 512):
        c = Case([100], 40, 4, 2, head_dim, seed=10)
        clean = Case([100], 40, 4, 2, head_dim, seed=10)
        c.q[0, 3, 1, 0] = float("nan")
        c.q[0, 20, 2, 9] = float("inf")
        got = c.device().call().cpu()[0].double()
        want, bound = clean.want(0)
        ok = torch.ones((40, 4), dtype=torch.bool)
        ok[3, 1] = ok[20, 2] = False
        assert ((got - want).abs() <= bound)[ok].all()
        assert got[3, 1].isnan().all()


@pytest.mark.parametrize("head_dim", [256, 512])
def test_rejected_requests_are_nan_and_reported(head_dim):
    c = Case([-1, 50, 300, 20], 20, 4, 2, head_dim, counts=[20, 21, 20, 20], seed=11)
    c.device()
    c.dt = c.table[:, :2].contiguous().cuda()      # room for 256 rows: request 2 does not fit
    out = c.call().cpu()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CONTEXT
    assert out[:3].isnan().all()
    want, bound = c.want(3)
    assert ((out[3].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("head_dim", [256, 512])
def test_a_page_outside_the_pool_reads_as_zeros_and_is_reported(head_dim):
    c = Case([200, 200], 30, 4, 2, head_dim, seed=12)
    c.device()
    c.dt[0, 0] = 1 << 20
    c.keys[0][:128] = 0
    c.values[0][:128] = 0
    out = c.call().cpu()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CACHE_ID
    for b in range(2):
        want, bound = c.want(b)
        assert ((out[b].double() - want).abs() <= bound).all(), b


def test_pages_that_nobody_sees_are_not_read():
    """Entries behind the window and past the keys hold ids of no page: no error."""
    for head_dim in (256, 512):
        c = Case([1000, 130], 5, 4, 2, head_dim, window=100, sinks=3, seed=13)
        c.device()
        c.dt[0, 1:7] = -1
        c.dt[1, 2:] = 1 << 20
        c.check(c.call())
        assert carat.carat_get_device_status(clear=True) == 0


def test_streams_graphs_and_repeats_give_the_same_bits():
    c = Case([3000, 77], 9, 16, 2, 512, window=2000, sinks=5, seed=14).device()
    first = c.call().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.out.fill_(7.0)
        c.call()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(first, c.out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    for _ in range(3):
        c.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, c.out)
    # the captured call follows what the device holds: other lengths and another table
    c.dc.copy_(torch.tensor([1500, 10], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    replayed = c.out.clone()
    c.out.fill_(7.0)
    assert torch.equal(replayed, c.call())


def test_two_calls_at_once_with_workspaces_of_their_own():
    cases = [Case([4000], 3, 16, 2, 512, seed=15).device(),
             Case([2000, 9], 2, 16, 8, 256, window=1024, sinks=4, seed=16).device()]
    alone = [c.call().clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                c.call()
    torch.cuda.synchronize()
    for a, c in zip(alone, cases):
        assert torch.equal(a, c.out)


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,window,counts", [
    (16, 8, 256, 700, None), (16, 2, 512, 0, [900, 41])])
def test_two_long_calls_at_once(q_heads, kv_heads, head_dim, window, counts):
    """More items than CTA pairs run at once, of two launches: whose work is taken over when
    depends on the other."""
    cases = [Case([0, 600], 900, q_heads, kv_heads, head_dim, window=window, sinks=9,
                  counts=counts, seed=s).device() for s in (21, 22)]
    alone = [c.call().clone() for c in cases]
    for c, out in zip(cases, alone):
        c.check(out, rows=[0, 1, 40, 127, 128, 500, 899])
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        for c in cases:
            c.out.fill_(7.0)
        torch.cuda.synchronize()
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                c.call()
        torch.cuda.synchronize()
        for a, c in zip(alone, cases):
            assert torch.equal(a, c.out)


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,ctx,k,counts", [
    (16, 2, 512, [3000, 10, 500], 200, None),             # more rows than CTAs merge at once
    (16, 2, 512, [3000, 10, 0, 700], 170, [170, 33, 0, 1]),
    (16, 8, 256, [5000, 0, 130, 2900], 150, [3, 150, 0, 149]),
    (8, 2, 256, [9, 7000, 64, 80, 300], 250, [250, 250, 1, 0, 129]),
    (16, 8, 256, [0, 1], 400, None)])                      # no request needs a second piece
def test_many_rows_in_pieces(q_heads, kv_heads, head_dim, ctx, k, counts):
    c = Case(ctx, k, q_heads, kv_heads, head_dim, counts=counts, seed=25, spread=2.0).device()
    assert c.ws is not None
    out = c.call()
    c.check(out, rows=[0, 1, 2, 15, 16, 31, 32, 63, 64, 127, 128, 148, 149, 169, 199, 249, 399])
    again = out.clone()
    c.out.fill_(7.0)
    assert torch.equal(c.call(), again)


@pytest.mark.parametrize("q_heads,kv_heads,head_dim", [(5, 1, 256), (16, 2, 512), (8, 1, 512)])
@pytest.mark.parametrize("per", [1, 2, 4, 5, 7, 8, 9, 40])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (130, 5), (600, 700)])
def test_as_many_pieces_as_tiles(q_heads, kv_heads, head_dim, per, window, sinks):
    """Tables of `per` pages of 128 keys, requests that fill them and others that do not."""
    for ctx in ([128 * per - 3], [128 * per - 3, 20, 0]):
        c = Case(ctx, 3, q_heads, kv_heads, head_dim, window=window, sinks=sinks, seed=per,
                 spread=2.0).device()
        assert c.table.shape[1] == per
        c.check(c.call())


def test_many_rows_in_pieces_with_a_rejected_request():
    c = Case([3000, 40, 200], 200, 16, 2, 512, seed=26)
    c.device()
    c.dc[1] = c.kp.shape[1] * c.table.shape[1]     # its new tokens do not fit
    out = c.call()
    assert out[1].isnan().all()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CONTEXT
    for b in (0, 2):
        for j in (0, 63, 64, 199):
            want, bound = c.want(b, [j])
            assert ((out[b, j].cpu().double() - want[0]).abs() <= bound[0]).all()


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,k", [(16, 8, 256, 130), (16, 2, 512, 130),
                                                         (16, 2, 512, 3)])
def test_views_that_begin_on_16_bytes(q_heads, kv_heads, head_dim, k):
    c = Case([300, 5], k, q_heads, kv_heads, head_dim, window=200, sinks=3, seed=23).device()
    want = c.call().clone()
    c.check(want)
    for name in ("dq", "dk", "dv", "out", "ws"):
        t = getattr(c, name)
        if t is None:
            continue
        buf = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
        at = -buf.data_ptr() % 32 // t.element_size() + 16 // t.element_size()
        view = buf[at:at + t.numel()].view(t.shape)
        view.copy_(t)
        assert view.data_ptr() % 32 == 16
        setattr(c, name, view)
    c.out.fill_(7.0)
    assert torch.equal(c.call(), want)


def test_a_call_reads_what_the_one_before_wrote():
    """Each call's queries are the outputs of the one before, nothing in between waits."""
    def chain(wait):
        c = Case([2000, 9], 4, 16, 2, 512, seed=24, spread=20.0).device()
        outs = []
        for _ in range(20):
            c.out = torch.empty_like(c.dq)
            c.call()
            if wait:
                torch.cuda.synchronize()
            outs.append(c.out)
            c.dq = c.out
        torch.cuda.synchronize()
        return outs
    for a, b in zip(chain(True), chain(False)):
        assert torch.equal(a, b)


def test_no_requests_and_bad_arguments():
    c = Case([10], 4, 4, 2, 256, seed=17).device()
    carat.carat_paged_chunk_attention(c.out[:0], c.dq[:0], c.dk, c.dv, c.dt[:0], c.dc[:0],
                                      scale=1.0)
    with pytest.raises(TypeError):
        carat.carat_paged_chunk_attention(c.out.float(), c.dq, c.dk, c.dv, c.dt, c.dc, scale=1.0)
    with pytest.raises(ValueError):
        carat.carat_paged_chunk_attention(c.out, c.dq, c.dk, c.dv, c.dt.cpu(), c.dc, scale=1.0)
    with pytest.raises(ValueError):
        carat.carat_paged_chunk_attention(c.out, c.dq.transpose(1, 2), c.dk, c.dv, c.dt, c.dc,
                                          scale=1.0)
    with pytest.raises(ValueError):
        carat.carat_paged_chunk_attention(c.out, c.dq, c.dk, c.dv, c.dt, c.dc[:0], scale=1.0)
    for kw in (dict(window=-1), dict(sinks=-1), dict(window=-(1 << 40))):
        with pytest.raises(carat.CaratError):
            carat.carat_paged_chunk_attention(c.out, c.dq, c.dk, c.dv, c.dt, c.dc, scale=1.0,
                                              workspace=c.ws, **kw)


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,ctx,k,window", [
    (16, 2, 512, [9000, 20000], 3, 0), (16, 8, 256, [9000, 20000], 3, 0),
    (16, 2, 512, [500, 90], 300, 0), (16, 8, 256, [500, 2000], 300, 700)])
def test_cold_and_warm_caches_give_the_same_bits(q_heads, kv_heads, head_dim, ctx, k, window):
    """Loads that come late from memory change the order in which the roles of a CTA pair
    meet, and nothing else."""
    c = Case(ctx, k, q_heads, kv_heads, head_dim, window=window, sinks=9, seed=18, spread=3.0,
             page_rows=384).device()
    first = c.call().clone()
    c.check(first, rows=[0, 1, 2, 151, 299])
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    for i in range(40):
        if i % 2:
            flush.fill_(i)
        c.out.fill_(7.0)
        c.call()
        assert torch.equal(first, c.out), i


@pytest.mark.parametrize("counts", [None, [2600, 3, 0, 17]])
def test_more_items_than_the_grid_has_cta_pairs(counts):
    """64 heads share a KV head: four tokens an item, 650 of them a request; with counts, most
    of a padded batch's CTA pairs find nothing to do."""
    ctx = [100] if counts is None else [100, 0, 7, 500]
    c = Case(ctx, 2600, 64, 1, 256, counts=counts, window=300, sinks=2, seed=19).device()
    c.check(c.call(), rows=[0, 1, 2, 3, 4, 16, 1000, 1503, 2431, 2432, 2433, 2598, 2599])


# Many requests of few rows take other ways through the library than one or two: at head_dim
# 512 the stream-K kernel (32 pairs of request and KV head, 16 without a window), else pieces
# whose number goes by the requests' lengths.
MANY = [(16, 2, 512, 17), (3, 1, 512, 33), (64, 4, 512, 9), (16, 8, 256, 5), (4, 1, 256, 40),
        (2, 1, 256, 2)]


def _ragged(n, longest, seed):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 300, (n,), generator=g).tolist()
    c[0], c[-1] = longest, 0
    if n > 2:
        c[1] = 127
    return c


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
@pytest.mark.parametrize("k", [1, 3])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 3), (128, 200), (513, 1 << 30)])
def test_many_requests(q_heads, kv_heads, head_dim, batch, k, window, sinks):
    c = Case(_ragged(batch, 2500, k), k, q_heads, kv_heads, head_dim, window=window, sinks=sinks,
             seed=20, spread=2.0, page_rows=256).device()
    c.check(c.call())


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
@pytest.mark.parametrize("window", [0, 70])
def test_many_requests_with_counts(q_heads, kv_heads, head_dim, batch, window):
    counts = [i % 5 for i in range(batch)]
    c = Case(_ragged(batch, 1000, 3), 4, q_heads, kv_heads, head_dim, counts=counts, window=window,
             sinks=5, seed=21).device()
    c.check(c.call())
    c = Case(_ragged(batch, 1000, 3), 4, q_heads, kv_heads, head_dim, counts=[0] * batch,
             window=window, seed=21).device()
    c.check(c.call())


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
def test_non_finite_values_among_many_requests(q_heads, kv_heads, head_dim, batch, window, bad):
    """In keys that some of a request's queries see: the newest but one, and one that the
    window leaves between the first query and the last; in the stale rows anyway."""
    k, ctx = 4, [200 + i for i in range(batch)]
    clean = Case(ctx, k, q_heads, kv_heads, head_dim, window=window, sinks=2, seed=22)
    c = Case(ctx, k, q_heads, kv_heads, head_dim, window=window, sinks=2, seed=22)
    hit = {0: ctx[0] + 2, batch - 1: ctx[-1] + 1 - window if window else ctx[-1] + 1}
    for b, t in hit.items():
        c.values[b][t, kv_heads - 1, 11] = bad
        c.keys[b][ctx[b] + k - 1, 0, 3] = bad
    c.write()
    got = c.device().call().cpu()
    g = q_heads // kv_heads
    for b in range(batch):
        want, bound = clean.want(b)
        for j in range(k):
            p = ctx[b] + j
            for h in range(q_heads):
                n = ctx[b] + k
                poisoned = b in hit and ((h // g == kv_heads - 1 and bool(
                    ref.seen(p, n, window, 2)[hit[b]])) or (h // g == 0 and j == k - 1))
                if not poisoned:
                    off = (got[b, j, h].double() - want[j, h]).abs()
                    assert (off <= bound[j, h]).all(), (b, j, h)
                elif not (h // g == 0 and j == k - 1):
                    assert not got[b, j, h, 11].isfinite(), (b, j, h)


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
def test_many_requests_some_rejected(q_heads, kv_heads, head_dim, batch):
    ctx = _ragged(batch, 400, 5)
    counts = [3] * batch
    c = Case(ctx, 3, q_heads, kv_heads, head_dim, counts=counts, seed=23).device()
    last = batch - 1
    c.dc[last] = -5
    if batch > 2:
        c.dn[2] = 4
        c.dc[1] = 1 << 30
    out = c.call().cpu()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CONTEXT
    rejected = {last, 1, 2} if batch > 2 else {last}
    for b in range(batch):
        if b in rejected:
            assert out[b].isnan().all(), b
        else:
            want, bound = c.want(b)
            assert ((out[b].double() - want).abs() <= bound).all(), b


@pytest.mark.parametrize("q_heads,kv_heads,head_dim,batch", MANY)
def test_many_requests_bad_pages_queries_and_repeats(q_heads, kv_heads, head_dim, batch):
    c = Case([300] * batch, 2, q_heads, kv_heads, head_dim, seed=24)
    clean = Case([300] * batch, 2, q_heads, kv_heads, head_dim, seed=24)
    c.q[0, 1, 0, 5] = float("nan")
    c.device()
    c.dt[batch - 1, 1] = -3
    for x in (clean.keys, clean.values):
        x[batch - 1][128:256] = 0
    first = c.call().clone()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CACHE_ID
    assert first[0, 1, 0].isnan().all()
    for b in range(batch):
        want, bound = clean.want(b)
        ok = torch.ones(want.shape[:2], dtype=torch.bool)
        if b == 0:
            ok[1, 0] = False
        assert (((first[b].cpu().double() - want).abs() <= bound)[ok]).all(), b
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    for i in range(12):
        flush.fill_(i)
        c.out.fill_(7.0)
        c.call()
        assert torch.equal(first.view(torch.int16), c.out.view(torch.int16)), i
    carat.carat_get_device_status(clear=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    c.out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), c.out.view(torch.int16))
    carat.carat_get_device_status(clear=True)
