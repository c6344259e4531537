"""Rotary paged appends against their definition in 64 bits, position by
position (GPU, through the C ABI).

Tolerances.  A rotated element is two fp32 products and a sum: off by at most
3 * 2^-24 (|x| + |partner|), written 2^-22 here.  A bf16 store adds 2^-8 of the
value, an e4m3 store 2^-4 of it or, for subnormals, 2^-10 of the scale.  Values
(V) are copied, or quantised from exact products: those have to be equal."""
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


class Setup:
    """A pool of pages with known contents, a page table in no order, and one
    step's rows.  Host copies of everything as it was before the call."""

    def __init__(self, ctx, k, q_heads, kv_heads, head_dim, *, rotary_dim=None, page_rows=128,
                 block_rows=0, seed=0, fused=False, counts=None, positions=None, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.k, self.B = list(ctx), k, len(ctx)
        self.hq, self.hkv, self.d = q_heads, kv_heads, head_dim
        self.page_rows, self.block_rows = page_rows, block_rows
        per = max(1, -(-max(max(c, 0) + k for c in ctx) // page_rows))
        self.num_pages = self.B * per + 2
        pool = (self.num_pages, page_rows, kv_heads, head_dim)
        if block_rows:
            def pages():
                x = (torch.randn(pool, generator=g) * 100).clamp(-448, 448)
                return x.to(ref.E4M3).view(torch.uint8)

            shape = (self.num_pages, page_rows // block_rows, kv_heads)
            self.ks = torch.exp2(torch.randint(-9, -4, shape, generator=g).float())
            self.vs = torch.exp2(torch.randint(-9, -4, shape, generator=g).float())
        else:
            def pages():
                return torch.randn(pool, generator=g).bfloat16()
        self.kp, self.vp = pages(), pages()
        perm = torch.randperm(self.num_pages, generator=g)[:self.B * per]
        self.table = perm.view(self.B, per).to(torch.int32)
        width = (q_heads + 2 * kv_heads) * head_dim
        qkv = (torch.randn((self.B, k, width), generator=g) * spread).bfloat16()
        nq, nk = q_heads * head_dim, kv_heads * head_dim
        parts = (qkv[..., :nq], qkv[..., nq:nq + nk], qkv[..., nq + nk:])
        dev = qkv.cuda()
        dparts = (dev[..., :nq], dev[..., nq:nq + nk], dev[..., nq + nk:])
        heads = (q_heads, kv_heads, kv_heads)
        self.q, self.kn, self.vn = (x.reshape(self.B, k, h, head_dim) for x, h in zip(parts, heads))
        d = [x.unflatten(-1, (h, head_dim)) if fused else
             x.contiguous().view(self.B, k, h, head_dim) for x, h in zip(dparts, heads)]
        self.dq, self.dkn, self.dvn = d
        self.r = rotary_dim or head_dim
        self.rows = per * page_rows
        self.cs = engine.rotary_table(self.rows, self.r, device="cpu")
        self.counts = counts
        self.positions = positions
        self.dkp, self.dvp, self.dtable = self.kp.cuda(), self.vp.cuda(), self.table.cuda()
        self.dcs = self.cs.cuda()
        if block_rows:
            self.dks, self.dvs = self.ks.cuda(), self.vs.cuda()
        self.q_out = torch.full((self.B, k, q_heads, head_dim), 7.0, dtype=torch.bfloat16,
                                device="cuda")

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def call(self, interleaved=False, queries=True, **kw):
        args = dict(cos_sin=self.dcs, interleaved=interleaved,
                    new_counts=None if self.counts is None else self.i32(self.counts),
                    positions=None if self.positions is None else self.i32(self.positions))
        if queries:
            args.update(queries=self.dq, queries_out=self.q_out)
        args.update(kw)
        ctx = self.i32(self.ctx)
        if self.block_rows:
            carat.carat_paged_rope_append_fp8(self.dkp, self.dvp, self.dks, self.dvs, self.dtable,
                                              self.dkn, self.dvn, ctx, **args)
        else:
            carat.carat_paged_rope_append(self.dkp, self.dvp, self.dtable, self.dkn, self.dvn, ctx,
                                          **args)
        torch.cuda.synchronize()

    def request_ok(self, b):
        n = self.k if self.counts is None else self.counts[b]
        return self.ctx[b] >= 0 and 0 <= n <= self.k and self.ctx[b] + n <= self.rows

    def pos(self, b, j):
        p = self.ctx[b] + j if self.positions is None else self.positions[b][j]
        return p if 0 <= p < self.cs.shape[0] else None

    def place(self, b, t):
        page = int(self.table[b, t // self.page_rows])
        return (page, t % self.page_rows) if 0 <= page < self.num_pages else None

    def check_queries(self, interleaved):
        got = self.q_out.cpu()
        for b in range(self.B):
            n = self.k if self.counts is None else self.counts[b]
            for j in range(self.k):
                if not self.request_ok(b) or (j < n and self.pos(b, j) is None):
                    assert got[b, j].isnan().all(), (b, j)
                elif j >= n:
                    assert (got[b, j] == 7.0).all(), (b, j)
                else:
                    x = self.q[b, j].double()
                    y = ref.rotate(x, self.cs, self.pos(b, j), interleaved)
                    tol = 2.0 ** -8 * y.abs() + 2.0 ** -22 * ref.pair_magnitude(x, self.cs,
                                                                                 interleaved)
                    assert ((got[b, j].double() - y).abs() <= tol).all(), (b, j)

    def check_bf16(self, interleaved):
        kp, vp = self.dkp.cpu(), self.dvp.cpu()
        ek, ev = self.kp.clone(), self.vp.clone()
        touched = torch.zeros(self.num_pages, self.page_rows, dtype=torch.bool)
        for b in range(self.B):
            if not self.request_ok(b):
                continue
            for j in range(self.k if self.counts is None else self.counts[b]):
                at = self.place(b, self.ctx[b] + j)
                if self.pos(b, j) is None or at is None:
                    continue
                ev[at] = self.vn[b, j]
                touched[at] = True
                x = self.kn[b, j].double()
                y = ref.rotate(x, self.cs, self.pos(b, j), interleaved)
                tol = 2.0 ** -8 * y.abs() + 2.0 ** -22 * ref.pair_magnitude(x, self.cs, interleaved)
                assert ((kp[at].double() - y).abs() <= tol).all(), (b, j)
        same = kp.view(torch.int16) == ek.view(torch.int16)
        assert same[~touched].all()
        assert torch.equal(vp.view(torch.int16), ev.view(torch.int16))

    def check_fp8(self, interleaved):
        R = self.block_rows
        kp, vp = self.dkp.cpu(), self.dvp.cpu()
        scales = (self.dks.cpu(), self.dvs.cpu())
        touched = torch.zeros(self.num_pages, self.page_rows, dtype=torch.bool)
        for b in range(self.B):
            if not self.request_ok(b):
                continue
            n = self.k if self.counts is None else self.counts[b]
            ctx = self.ctx[b]
            for t0 in range(ctx // R * R, ctx + n, R):
                rows = [t for t in range(max(t0, ctx), min(t0 + R, ctx + n))
                        if self.pos(b, t - ctx) is not None]
                at0 = self.place(b, t0)
                if not rows or at0 is None:
                    continue
                page, r0 = at0
                for is_v, (pages, before, after, new) in enumerate((
                        (kp, self.kp, scales[0], self.kn), (vp, self.vp, scales[1], self.vn))):
                    x = torch.stack([new[b, t - ctx].double() for t in rows])
                    mag = torch.zeros_like(x)
                    if not is_v:
                        mag = torch.stack([ref.pair_magnitude(y, self.cs, interleaved) for y in x])
                        x = torch.stack([ref.rotate(y, self.cs, self.pos(b, t - ctx), interleaved)
                                         for y, t in zip(x, rows)])
                    old = (self.ks, self.vs)[is_v][page, r0 // R].double()
                    for h in range(self.hkv):
                        fin = torch.where(x[:, h].isfinite(), x[:, h].abs(), 0.0)
                        # an amax within its own rounding of a border may go either way
                        amax = float(fin.max())
                        slack = 2.0 ** -21 if not is_v else 0.0
                        wants = {max(2.0 ** ref.scale_exponent(a), 0.0 if t0 >= ctx else float(old[h]))
                                 for a in (amax * (1 - slack), amax * (1 + slack))}
                        s = float(after[page, r0 // R, h])
                        assert s in wants, (b, t0, h, is_v, s, wants)
                        for i, t in enumerate(rows):
                            got = ref.decode(pages[page, r0 + t - t0, h])
                            y = x[i, h] / s
                            if is_v:
                                want = (x[i, h] / s).float().clamp(-448, 448).to(ref.E4M3)
                                w8, g8 = want.view(torch.uint8), pages[page, r0 + t - t0, h]
                                nan = x[i, h].isnan()
                                assert torch.equal(w8[~nan], g8[~nan]), (b, t, h)
                                assert ref.decode(g8)[nan].isnan().all()
                            else:
                                tol = torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10)
                                                    .double()) + 2.0 ** -21 * mag[i, h] / s
                                ok = (got - y.clamp(-448, 448)).abs() <= tol
                                assert (ok | y.isnan()).all(), (b, t, h)
                        for t in range(t0, ctx):
                            was = before[page, r0 + t - t0, h]
                            want = (ref.decode(was) * (float(old[h]) / s)).float().to(ref.E4M3)
                            g8 = pages[page, r0 + t - t0, h]
                            assert torch.equal(want.view(torch.uint8), g8), (b, t, h, is_v)
                for t in range(t0, ctx):
                    touched[page, r0 + t - t0] = True
                for t in rows:
                    touched[page, r0 + t - t0] = True
        for got, was in ((kp, self.kp), (vp, self.vp)):
            assert torch.equal(got[~touched], was[~touched])

    def check(self, interleaved=False, queries=True):
        if queries:
            self.check_queries(interleaved)
        if self.block_rows:
            self.check_fp8(interleaved)
        else:
            self.check_bf16(interleaved)


SHAPES = {
    # ctx, k, Hq, Hkv, D, keywords
    "one_token": ([0], 1, 16, 2, 512, {}),
    "decode": ([0, 1, 127, 128, 700], 1, 16, 8, 256, {}),
    "verify": ([5, 126, 127, 128, 900], 4, 16, 2, 512, {"fused": True}),
    "sixteen": ([0, 113, 250], 16, 8, 1, 256, {"rotary_dim": 64}),
    "ragged": ([0, 3, 130, 60], 70, 4, 2, 256, {"counts": [70, 0, 1, 69], "fused": True}),
    "odd_heads": ([10, 255], 3, 5, 5, 48, {"rotary_dim": 16}),
    "narrow": ([31, 32, 33], 5, 3, 1, 16, {}),
    "wide": ([100], 9, 2, 2, 1024, {"rotary_dim": 256}),
    "d160": ([17, 90], 33, 4, 2, 160, {"rotary_dim": 96, "page_rows": 256}),
    "prompt": ([0, 200], 300, 4, 1, 512, {"page_rows": 384}),
}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("block_rows", [0, 16, 32, 64, 128])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_append_matches_the_definition(shape, block_rows, interleaved):
    ctx, k, hq, hkv, d, kw = SHAPES[shape]
    s = Setup(ctx, k, hq, hkv, d, block_rows=block_rows, seed=len(shape) + block_rows, **kw)
    s.call(interleaved)
    s.check(interleaved)
    assert carat.carat_get_device_status(clear=True) == 0


@pytest.mark.parametrize("block_rows", [0, 32])
def test_keys_and_values_only(block_rows):
    s = Setup([40, 100], 6, 4, 2, 256, block_rows=block_rows, seed=3)
    s.call(queries=False)
    s.check(queries=False)
    assert (s.q_out == 7.0).all()


@pytest.mark.parametrize("block_rows", [0, 16])
def test_explicit_positions_turn_the_angle_only(block_rows):
    """A token tree: siblings share a position; storage rows stay in order."""
    s = Setup([50, 3], 5, 4, 2, 256, block_rows=block_rows, seed=4,
              positions=[[50, 51, 51, 51, 52], [3, 4, 5, 4, 5]])
    s.call()
    s.check()


@pytest.mark.parametrize("block_rows", [0, 16])
def test_rejected_requests_and_tokens(block_rows):
    """Bad lengths, counts, positions and pages are skipped and reported; every
    other byte stays or is written as usual."""
    s = Setup([10, -1, 20, 100, 30, 126], 4, 4, 2, 256, block_rows=block_rows, seed=5,
              counts=[4, 4, 5, 4, -1, 4],
              positions=[[10, -1, 12, 4000], [0] * 4, [20] * 4, [100, 101, 102, 103], [0] * 4,
                         [126, 127, 128, 129]])
    assert s.rows == 256
    s.table[5, 1] = s.num_pages          # position 128's page lies outside the pool
    s.dtable = s.table.cuda()
    s.call()
    s.check()
    status = carat.carat_get_device_status(clear=True)
    assert status == (carat.CARAT_DEV_BAD_CONTEXT | carat.CARAT_DEV_BAD_POSITION |
                      carat.CARAT_DEV_BAD_CACHE_ID)


@pytest.mark.parametrize("block_rows", [0, 16])
def test_the_last_row_of_the_capacity(block_rows):
    s = Setup([124], 4, 2, 2, 256, block_rows=block_rows, seed=6)
    assert s.rows == 128
    s.call()
    s.check()
    assert carat.carat_get_device_status(clear=True) == 0
    s2 = Setup([124], 4, 2, 2, 256, block_rows=block_rows, seed=6)
    s2.ctx = [125]
    s2.call()
    s2.check()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CONTEXT


@pytest.mark.parametrize("block_rows", [0, 64])
def test_in_place_queries(block_rows):
    s = Setup([7, 77], 4, 8, 2, 256, block_rows=block_rows, seed=8)
    keep = s.dq.clone()
    s.call()
    want = s.q_out.clone()
    s.call(queries_out=s.dq)
    assert torch.equal(s.dq.view(torch.int16), want.view(torch.int16))
    assert not torch.equal(keep, s.dq)


@pytest.mark.parametrize("spread", [2.0 ** -115, 1e-6, 0.0, 1e4, 3e38])
def test_scales_over_the_whole_range(spread):
    """Tiny, zero and huge rows: the exponent is kept in [-100, 100]."""
    s = Setup([0, 20], 20, 2, 2, 256, block_rows=16, seed=9, spread=spread)
    assert s.kn.isfinite().all() or spread == 3e38
    if spread == 3e38:
        for t in (s.kn, s.vn, s.q):
            t.clamp_(-2.0 ** 126, 2.0 ** 126)
        s.dkn, s.dvn, s.dq = s.kn.cuda(), s.vn.cuda(), s.q.cuda()
    s.call()
    s.check_fp8(False)


def test_infinities_and_nan_do_not_reach_the_scale():
    """V: an infinity is stored as the largest magnitude, a NaN as NaN, and the
    block's other values keep the scale they would have had."""
    s = Setup([16], 16, 2, 2, 256, block_rows=16, seed=10)
    clean = Setup([16], 16, 2, 2, 256, block_rows=16, seed=10)
    s.vn[0, 3, 1, 5] = float("inf")
    s.vn[0, 4, 0, 9] = float("nan")
    s.vn[0, 5, 1, 6] = -float("inf")
    s.dvn = s.vn.cuda()
    s.call()
    clean.call()
    assert torch.equal(s.dvs, clean.dvs)
    page, r0 = s.place(0, 16)
    got = ref.decode(s.dvp.cpu()[page])
    assert got[r0 + 3, 1, 5] == 448 and got[r0 + 5, 1, 6] == -448 and got[r0 + 4, 0, 9].isnan()
    a, b = s.dvp.clone(), clean.dvp.clone()
    for x in (a, b):
        for at in ((3, 1, 5), (4, 0, 9), (5, 1, 6)):
            x[page, r0 + at[0], at[1], at[2]] = 0
    assert torch.equal(a, b)


def test_a_block_grows_its_scale_token_by_token():
    """Sixteen one-token appends, each larger than the last: the block's scale
    doubles again and again and every row ends at the last scale's rounding."""
    s = Setup([16], 1, 2, 1, 256, block_rows=16, seed=11)
    page, r0 = s.place(0, 16)
    want = torch.zeros(16, 256, dtype=torch.float64)
    scale = None
    g = torch.Generator().manual_seed(12)
    for i in range(16):
        x = (torch.randn((1, 1, 1, 256), generator=g) * 1.9 ** i).bfloat16()
        s.dkn = s.dvn = x.cuda()
        s.ctx = [16 + i]
        s.call(queries=False)
        need = 2.0 ** ref.scale_exponent(float(x.abs().max()))
        new = need if scale is None else max(scale, need)
        if scale is not None:
            want = (want * (scale / new)).float().to(ref.E4M3).float().double()
        scale = new
        want[i] = (x.double().flatten() / scale).float().to(ref.E4M3).float().double()
        assert float(s.dvs[page, r0 // 16, 0]) == scale
    got = ref.decode(s.dvp.cpu()[page, r0:r0 + 16, 0])
    assert torch.equal(got, want)


@pytest.mark.parametrize("block_rows", [0, 16])
def test_captured_and_replayed(block_rows):
    s = Setup([30, 100], 4, 8, 2, 256, block_rows=block_rows, seed=13)
    ctx = s.i32(s.ctx)
    args = dict(cos_sin=s.dcs, queries=s.dq, queries_out=s.q_out)

    def call(stream):
        if block_rows:
            carat.carat_paged_rope_append_fp8(s.dkp, s.dvp, s.dks, s.dvs, s.dtable, s.dkn, s.dvn,
                                              ctx, stream=stream, **args)
        else:
            carat.carat_paged_rope_append(s.dkp, s.dvp, s.dtable, s.dkn, s.dvn, ctx, stream=stream,
                                          **args)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call(side)
    assert (s.q_out == 7.0).all()
    graph.replay()
    torch.cuda.synchronize()
    s.check()


def test_binding_refuses_what_would_fault():
    s = Setup([3, 5], 4, 4, 2, 256, block_rows=16, seed=14)
    ok = dict(cos_sin=s.dcs)
    pos = (s.dkp, s.dvp, s.dks, s.dvs, s.dtable, s.dkn, s.dvn, s.i32([3, 5]))

    def refused(error, *, at=None, value=None, **kw):
        args = list(pos)
        if at is not None:
            args[at] = value
        with pytest.raises(error):
            carat.carat_paged_rope_append_fp8(*args, **{**ok, **kw})

    refused(TypeError, at=0, value=s.dkp.view(torch.int8))
    refused(ValueError, at=1, value=s.dvp[:-1])
    refused(ValueError, at=2, value=s.dks[:, :-1])
    refused(ValueError, at=4, value=s.dtable[:1])
    refused(ValueError, at=4, value=s.dtable.cpu())
    refused(ValueError, at=5, value=s.dkn.transpose(2, 3))
    refused(ValueError, at=6, value=s.dvn[:, :3])
    refused(ValueError, at=7, value=s.i32([3]))
    refused(ValueError, queries=s.dq)
    refused(ValueError, queries=s.dq, queries_out=s.q_out[..., :128])
    refused(TypeError, cos_sin=s.dcs.double())
    refused(ValueError, cos_sin=s.dcs.cpu())
    refused(carat.CaratError, cos_sin=s.dcs[:, :24].contiguous())       # rotary_dim 24
    refused(ValueError, positions=s.i32([1, 2]))
    refused(ValueError, new_counts=s.i32([1]))
    torch.cuda.synchronize()


@pytest.mark.parametrize("block_rows", [0, 32])
def test_offsets_past_32_bits(block_rows):
    """Pages behind the pool's 2^32-th element and tokens 2^28 elements apart: the
    same bytes as from a small pool and dense tokens."""
    B, k, hkv, d = 1, 17, 8, 512
    g = torch.Generator().manual_seed(31)
    dense = [torch.randn((B, k, hkv, d), generator=g).bfloat16().cuda() for _ in range(2)]
    stride = 1 << 28
    far = torch.empty((k - 1) * stride + 2 * hkv * d, dtype=torch.bfloat16, device="cuda")
    wide = [far[i * hkv * d:].as_strided((B, k, hkv, d), (k * stride, stride, d, 1))
            for i in range(2)]
    for x, y in zip(wide, dense):
        x.copy_(y)
    cs = engine.rotary_table(512, d)
    ctx = torch.tensor([120], dtype=torch.int32, device="cuda")
    many = (1 << 32) // (hkv * d) // 128 + 4
    got = []
    for pages, first, (kn, vn) in ((4, 0, dense), (many, many - 4, wide)):
        table = torch.tensor([[first + 3, first + 1]], dtype=torch.int32, device="cuda")
        dtype = torch.uint8 if block_rows else torch.bfloat16
        kp, vp = (torch.empty((pages, 128, hkv, d), dtype=dtype, device="cuda") for _ in range(2))
        for x in (kp, vp):
            x[table[0].long()] = 0
        if block_rows:
            ks, vs = (torch.ones((pages, 128 // block_rows, hkv), device="cuda") for _ in range(2))
            carat.carat_paged_rope_append_fp8(kp, vp, ks, vs, table, kn, vn, ctx, cos_sin=cs)
            got.append([x[table[0].long()].clone() for x in (kp, vp, ks, vs)])
        else:
            carat.carat_paged_rope_append(kp, vp, table, kn, vn, ctx, cos_sin=cs)
            got.append([x[table[0].long()].view(torch.int16).clone() for x in (kp, vp)])
        del kp, vp
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == 0
    for x, y in zip(*got):
        assert torch.equal(x, y) and (x != 0).any()
