"""A prompt in chunks, beams forked from it, decode steps under a window with first tokens,
pages freed behind the window and the pool compacted: the operators as an engine strings
them together, each output against 64 bits over a host-side history (GPU)."""
import pytest
import torch

import chunk_reference as ref
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


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Model:
    """One layer's requests with their tokens' keys and values (as stored) on the host."""

    def __init__(self, layer, table, history):
        self.layer, self.table, self.history = layer, table, history

    def stored(self, b, n):
        """Rows [0, n) of request b, by the layer's own table; NaN for pages given back."""
        rows = self.layer.page_rows
        out = []
        for pages in (self.layer.key_pages, self.layer.value_pages):
            flat = pages.cpu()
            ids = self.layer.page_table[b, :-(-n // rows)].tolist()
            out.append(torch.cat([flat[i] if i >= 0 else torch.full_like(flat[0], float("nan"))
                                  for i in ids])[:n])
        return out

    def follow(self, b, ctx, n):
        """Adds what was appended, and checks that what was there is as it was."""
        k, v = self.stored(b, ctx + n)
        first, end = self.layer.hidden(ctx)
        for new, old in zip((k, v), self.history[b]):
            for t0 in range(0, ctx, self.layer.page_rows):
                page = t0 // self.layer.page_rows
                if not first <= page < end:
                    t1 = min(ctx, t0 + self.layer.page_rows)
                    assert torch.equal(new[t0:t1].view(torch.int16), old[t0:t1].view(torch.int16))
        self.history[b] = [torch.cat([old[:ctx], new[ctx:]])
                           for new, old in zip((k, v), self.history[b])]

    def check(self, out, ctx, counts):
        q = self.layer.rotated[:out.numel()].view(out.shape).cpu().double()
        for b, n in enumerate(counts):
            if n == 0:
                continue
            self.follow(b, ctx[b], n)
            k, v = (x.double() for x in self.history[b])
            for j in sorted({0, n // 3, n - 1}):
                want, bound = ref.attention(q[b, j:j + 1], k, v, ctx[b] + j, self.layer.window,
                                            self.layer.sinks, self.layer.scale)
                off = (out[b, j].cpu().double() - want[0]).abs()
                assert (off <= bound[0]).all(), (b, j, float((off - bound[0]).max()))


@pytest.mark.parametrize("q_heads,kv_heads,head_dim", [(8, 4, 256), (16, 2, 512)])
@pytest.mark.parametrize("window,sinks", [(300, 3), (0, 0), (140, 150)])
def test_prompt_beams_steps_and_compaction(q_heads, kv_heads, head_dim, window, sinks):
    g = torch.Generator(device="cuda").manual_seed(31)

    def rows(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    lines, per = 2, 12
    pool = engine.SharedPool(num_pages=72, page_bytes=128 * kv_heads * head_dim * 2,
                             pages_per_ring=4, fill=float("nan"))
    cs = engine.rotary_table(per * 128, head_dim)
    common = dict(q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, cos_sin=cs, window=window,
                  sinks=sinks, max_proposals=4)
    table = torch.full((lines, per), -1, dtype=torch.int32)
    for b, n in enumerate((6, 4)):
        table[b, :n] = torch.tensor(pool.alloc.alloc_pages(n), dtype=torch.int32)
    layer = engine.PagedGlobalLayer(pool, table.cuda(), max_chunk=400, **common)
    model = Model(layer, table, [[torch.empty((0, kv_heads, head_dim), dtype=torch.bfloat16)] * 2
                                 for _ in range(lines)])

    # two prompts, in two chunks of different lengths
    ctx = [0, 0]
    for counts in ([400, 150], [297, 0]):
        k = max(counts)
        out = layer.chunk(rows(lines, k, q_heads, head_dim), rows(lines, k, kv_heads, head_dim),
                          rows(lines, k, kv_heads, head_dim), i32(ctx), new_counts=i32(counts))
        model.check(out, ctx, counts)
        ctx = [c + n for c, n in zip(ctx, counts)]

    # three beams: two of the first prompt (one goes on in its page), one of the second
    parents, children = [0, 1, 0], 3
    fresh = pool.alloc.alloc_pages(2)
    new_pages = [fresh[0], fresh[1], -1]
    child = torch.full((children, per), -1, dtype=torch.int32, device="cuda")
    lengths = i32([0] * children)
    layer.fork(i32(ctx), child, i32(parents), i32(new_pages), child_lengths=lengths)
    assert pool.alloc.share_pages(table[0, :ctx[0] // 128].tolist())
    ctx = [ctx[p] for p in parents]
    assert lengths.tolist() == ctx
    beams = engine.PagedGlobalLayer(pool, child, max_chunk=4, **common)
    with pytest.raises(ValueError):
        beams.chunk(rows(children, 5, q_heads, head_dim), None, None, i32(ctx))
    model = Model(beams, child, [list(model.history[p]) for p in parents])

    # decode and verify steps; pages behind the window are given back on the way
    for step, k in enumerate((1, 4, 3, 1)):
        for b in range(children):
            last = (ctx[b] + k - 1) // 128
            if child[b, last] < 0:
                child[b, last] = pool.alloc.alloc_pages(1)[0]
        args = (rows(children, k, q_heads, head_dim), rows(children, k, kv_heads, head_dim),
                rows(children, k, kv_heads, head_dim), i32(ctx))
        if window:
            out = beams.step(*args)
        else:
            out = beams.chunk(*args)
        model.check(out, ctx, [k] * children)
        ctx = [c + k for c in ctx]
        freed = 0
        for b in range(children):
            first, end = beams.hidden(ctx[b])
            ids = [i for i in child[b, first:end].tolist() if i >= 0]
            assert pool.alloc.free_pages(ids)
            child[b, first:end] = -1
            freed += len(ids)
        if step == 0:
            assert bool(freed) == bool(window)

        # other users of the pool come and go, and leave it in pieces
        other = pool.alloc.alloc_pages(24)
        assert pool.alloc.free_pages(other[::2])
        before = pool.alloc.stats()["whole_free_blocks"]
        moved = pool.compact([beams], 100)
        assert pool.alloc.stats()["whole_free_blocks"] >= before
        assert step or moved
        # those pages may have moved: theirs are the ones that no line names
        named = {i for i in child.flatten().tolist() if i >= 0}
        mine = [i for i in range(pool.num_pages) if i not in named and pool.alloc.share_pages([i])]
        for i in mine:
            while pool.alloc.free_pages([i]):
                pass


def test_forked_e4m3_caches_go_on_as_their_parent_does():
    g = torch.Generator(device="cuda").manual_seed(32)

    def rows(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    pool = engine.SharedPool(num_pages=12, page_bytes=128 * 2 * 512 * 2, pages_per_ring=4)
    cs = engine.rotary_table(1024, 512)
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    table[0, :2] = i32(pool.alloc.alloc_pages(2))
    layer = engine.Fp8PagedLayer(pool, table, cs, block_rows=32)
    assert layer.page_rows == 256
    n = 300
    layer.append(rows(1, n, 2, 512), rows(1, n, 2, 512), i32([0]))
    child = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    layer.fork(i32([n]), child, i32([0, 0]), i32(pool.alloc.alloc_pages(2)))
    beams = engine.Fp8PagedLayer(pool, child, cs, block_rows=32)
    beams.k_scales, beams.v_scales = layer.k_scales, layer.v_scales
    q, kn, vn = rows(1, 4, 16, 512), rows(1, 4, 2, 512), rows(1, 4, 2, 512)
    want = layer.step(q, kn, vn, i32([n]))
    got = beams.step(q.expand(2, -1, -1, -1).contiguous(), kn.expand(2, -1, -1, -1).contiguous(),
                     vn.expand(2, -1, -1, -1).contiguous(), i32([n, n]))
    # (the attention's pieces may be cut elsewhere: bf16 outputs, half a step apart)
    for b in range(2):
        off = (got[b].float() - want[0].float()).abs()
        assert (off <= 2.0 ** -7 * want[0].float().abs() + 2.0 ** -9).all()
        for x in (layer.k_scales, layer.v_scales):
            assert torch.equal(x[child[b, 1].long()], x[table[0, 1].long()])
        for x in (layer.key_pages, layer.value_pages):
            assert torch.equal(x[child[b, 1].long(), :n + 4 - 256], x[table[0, 1].long(), :n + 4 - 256])


def test_a_captured_decode_step_over_a_windowed_layer():
    g = torch.Generator(device="cuda").manual_seed(33)

    def rows(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    pool = engine.SharedPool(num_pages=16, page_bytes=128 * 8 * 256 * 2, pages_per_ring=4)
    table = torch.tensor([pool.alloc.alloc_pages(4) for _ in range(2)], dtype=torch.int32).cuda()
    layer = engine.PagedGlobalLayer(pool, table, q_heads=16, kv_heads=8, head_dim=256,
                                    cos_sin=engine.rotary_table(512, 256), window=128, sinks=4,
                                    max_proposals=2, max_chunk=300)
    layer.chunk(rows(2, 300, 16, 256), rows(2, 300, 8, 256), rows(2, 300, 8, 256), i32([0, 0]))
    inputs = (rows(2, 2, 16, 256), rows(2, 2, 8, 256), rows(2, 2, 8, 256), i32([300, 290]))
    step = engine.DecodeStep([layer], [inputs])
    assert step.outputs[0].dtype == torch.bfloat16
    eager = step.run()[0].clone()
    step.capture()
    step.outputs[0].zero_()
    assert torch.equal(step.replay()[0], eager)
    inputs[3].copy_(i32([310, 5]))
    replayed = step.replay()[0].clone()
    assert not torch.equal(replayed, eager)
    assert torch.equal(step.run()[0], replayed)


@pytest.mark.parametrize("raw", [False, True])
def test_a_compaction_on_another_stream_keeps_its_lists(raw):
    """Lists of the same size are made while the moves still wait on their stream (what they
    hold, -1, would move nothing)."""
    pool = engine.SharedPool(num_pages=64, page_bytes=128 * 2 * 256 * 2, pages_per_ring=4, fill=None)
    pool.k.view(torch.int16).copy_(torch.arange(64, device="cuda").repeat_interleave(
        pool.page_bytes // 2))
    pool.v.copy_(pool.k)
    pages = pool.alloc.alloc_pages(40)
    assert pool.alloc.free_pages([p for i, p in enumerate(pages) if i % 4 != 1])
    kept = pages[1::4]
    layer = engine.PagedGlobalLayer(pool, i32([kept]), q_heads=4, kv_heads=2, head_dim=256,
                                    max_chunk=4)
    slow = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(100):
            slow.copy_(slow.flip(0))
    moved = pool.compact([layer], 100, stream=side.cuda_stream if raw else side)
    assert moved > 0
    others = [i32([-1] * moved) for _ in range(64)]
    torch.cuda.synchronize()
    assert len(others) == 64
    table = layer.page_table[0].tolist()
    assert sum(a != b for a, b in zip(table, kept)) == moved
    held = pool.k.view(torch.int16).view(64, -1)[:, 0].tolist()
    assert [held[t] for t in table] == kept
