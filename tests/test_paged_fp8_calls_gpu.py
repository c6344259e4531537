"""Calls of the attention over e4m3 pages that its schedule treats apart: more
requests than the range search keeps counts of, one long request among short ones;
and refusals of numbers that do not fit an int (GPU, against 64 bits)."""
import pytest
import torch

from sliding_window_gqa_ring_gb300 import carat, engine
from test_paged_fp8_attention_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    carat.library()
    carat.carat_get_device_status(clear=True)
    yield
    assert carat.carat_get_device_status(clear=True) == 0


@pytest.mark.parametrize("kw,batch", [(dict(k=1, q_heads=2, kv_heads=1, head_dim=256), 1100),
                                      (dict(k=3, q_heads=4, kv_heads=1, head_dim=256), 1700),
                                      (dict(k=2, q_heads=8, kv_heads=2, head_dim=512), 2100)])
def test_more_requests_than_kept_tile_counts(kw, batch):
    """The range search keeps 1024, 1536 and 2048 requests' tile counts in shared
    memory and reads those of the others again; empty and rejected requests lie on
    both sides."""
    kept = {1100: 1024, 1700: 1536, 2100: 2048}[batch]
    k = kw["k"]
    n = [k + (i * 37) % 280 for i in range(batch)]
    for b in (0, kept - 1, kept, batch - 1):
        n[b] = 400 + b % 7
    c = Case(n, seed=71, **kw)
    ctx, counts = c.ctx.clone(), torch.full_like(c.ctx, k)
    rejected = set(range(5, batch, 50)) | {kept - 2, kept + 1}
    empty = set(range(7, batch, 50)) | {kept - 3, kept + 2}
    empty -= rejected
    ctx[sorted(rejected)] = -3
    counts[sorted(empty)] = 0
    out = c.call(ctx=ctx, counts=counts)
    torch.cuda.synchronize()
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CONTEXT
    c.check(out, [b for b in range(batch) if b not in rejected | empty])
    assert all(out[b].isnan().all() for b in rejected)
    assert all((out[b] == 3.0).all() for b in empty)


@pytest.mark.parametrize("kw", [dict(k=4, q_heads=16, kv_heads=2, head_dim=512),
                                dict(k=1, q_heads=16, kv_heads=8, head_dim=256),
                                dict(k=15, q_heads=16, kv_heads=2, head_dim=512)])
@pytest.mark.parametrize("at", [0, 31, 63])
def test_one_long_request_among_short_ones(kw, at):
    """It is cut into many times more pieces than the average that the merge's shape
    is chosen by."""
    n = [kw["k"] + (i * 13) % 100 for i in range(64)]
    n[at] = 9001
    Case(n, seed=72, **kw).run()


@pytest.mark.parametrize("window", [-1, -2 ** 31 - 5, -2 ** 32 + 5, -2 ** 63])
def test_negative_windows_are_refused_whatever_their_size(window):
    c = Case([100], 1, 4, 2, 256, seed=73)
    c.window = window
    with pytest.raises(carat.CaratError) as e:
        c.call()
    assert e.value.status == carat.CARAT_ERR_INVALID_ARG


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 3, 2 ** 70])
def test_windows_past_every_length_are_no_window(window):
    c = Case([300, 1], 1, 4, 2, 256, seed=74)
    first = c.run()
    c.window = window
    assert torch.equal(c.call().view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("captured", [False, True])
def test_a_step_whose_inputs_come_from_two_other_streams(captured):
    """Lengths written on one stream, keys and values on another, both joined before
    the step: its launches, which may start while the one before them drains, start
    behind both."""
    B, k, hq, hkv, d = 6, 4, 16, 2, 512
    g = torch.Generator().manual_seed(75)
    cs = engine.rotary_table(1024, d)
    new = [[torch.randn((B, k, h, d), generator=g).bfloat16().cuda() for h in (hq, hkv, hkv)]
           for _ in range(12)]
    first = torch.randn((B, 300, hkv, d), generator=g).bfloat16().cuda()
    start = torch.tensor([300 - 40 * b for b in range(B)], dtype=torch.int32, device="cuda")
    heavy = torch.randn((4096, 4096), device="cuda")

    def layer():
        pool = engine.SharedPool(num_pages=24, page_bytes=128 * hkv * d * 2, pages_per_ring=4,
                                 fill=0.0)
        table = torch.tensor([pool.alloc.alloc_pages(3) for _ in range(B)], dtype=torch.int32)
        made = engine.Fp8PagedLayer(pool, table.cuda(), cs, q_heads=hq, kv_heads=hkv, head_dim=d,
                                    max_proposals=k)
        made.append(first, first, torch.zeros_like(start), new_counts=start)
        return made

    plain = layer()
    want = []
    for i, (q, kn, vn) in enumerate(new):
        want.append(plain.step(q, kn, vn, start + 3 * i))
    torch.cuda.synchronize()

    joined = layer()
    q, kn, vn = (torch.zeros_like(x) for x in new[0])
    ctx, step = torch.zeros_like(start), torch.zeros_like(start)
    source = [torch.stack([n[j] for n in new]) for j in range(3)]
    which = torch.zeros(1, dtype=torch.int64, device="cuda")
    out = torch.empty_like(q)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]

    def run(stream):
        forks = torch.cuda.Event()
        forks.record(stream)
        for s in sides:
            s.wait_event(forks)
        with torch.cuda.stream(sides[0]):
            torch.mm(heavy, heavy)                  # late
            ctx.copy_(start + 3 * step)
        with torch.cuda.stream(sides[1]):
            torch.mm(heavy, heavy)
            for dst, src in zip((q, kn, vn), source):
                dst.copy_(src.index_select(0, which)[0])
        for s in sides:
            e = torch.cuda.Event()
            e.record(s)
            stream.wait_event(e)
        joined.step(q, kn, vn, ctx, out=out, stream=stream)

    stream = torch.cuda.Stream()
    run(stream)                                     # step 0 twice over: the same rows
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            run(stream)
    got = []
    for i in range(len(new)):
        which.fill_(i), step.fill_(i)
        torch.cuda.synchronize()
        graph.replay() if captured else run(stream)
        torch.cuda.synchronize()
        got.append(out.clone())
    assert carat.carat_get_device_status(clear=True) == 0
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
