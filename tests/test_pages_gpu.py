"""Copying, forking and moving pages against the same on the host, bit for bit (GPU)."""
import random

import pytest
import torch

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


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Pool:
    """Random bytes (NaNs among them) in pages and scales, on the host and the device."""

    def __init__(self, num_pages, page_rows, kv_heads, head_dim, block_rows=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        shape = (num_pages, page_rows, kv_heads, head_dim)
        bytes_ = 1 if block_rows else 2

        def pages():
            x = torch.randint(0, 256, (*shape[:3], head_dim * bytes_), generator=g,
                              dtype=torch.int16).to(torch.uint8)
            return x if block_rows else x.view(torch.bfloat16)

        self.host = [pages(), pages()]
        self.R = block_rows
        if block_rows:
            blocks = (num_pages, page_rows // block_rows, kv_heads)
            self.host += [torch.randn(blocks, generator=g) for _ in range(2)]
        self.dev = [x.cuda() for x in self.host]
        self.rows = page_rows

    def copy(self, a, b, n):
        for x in self.host[:2]:
            x[b, :n] = x[a, :n].clone()
        for x in self.host[2:]:
            x[b, :-(-n // self.R)] = x[a, :-(-n // self.R)].clone()

    def scales(self):
        return {"k_scales": self.dev[2], "v_scales": self.dev[3]} if self.R else {}

    def check(self):
        for h, d in zip(self.host, self.dev):
            bits = torch.int32 if h.dtype == torch.float32 else torch.uint8
            assert torch.equal(h.view(bits), d.cpu().view(bits))


SHAPES = [(128, 2, 512, 0), (128, 1, 8, 0), (256, 8, 256, 0), (128, 2, 512, 16), (256, 3, 256, 64),
          (384, 1, 16, 128)]


@pytest.mark.parametrize("page_rows,kv_heads,head_dim,block_rows", SHAPES)
@pytest.mark.parametrize("count,partial", [(1, False), (5, True), (40, True)])
def test_copy(count, partial, page_rows, kv_heads, head_dim, block_rows):
    pool = Pool(2 * count + 3, page_rows, kv_heads, head_dim, block_rows, seed=count)
    r = random.Random(count)
    ids = r.sample(range(2 * count + 3), 2 * count)
    src, dst = ids[:count], ids[count:]
    rows = [r.choice([0, 1, 15, 16, 17, page_rows - 1, page_rows, r.randint(0, page_rows)])
            for _ in src] if partial else None
    carat.carat_pages_copy(pool.dev[0], pool.dev[1], i32(src), i32(dst),
                           rows=i32(rows) if partial else None, **pool.scales())
    for i, (a, b) in enumerate(zip(src, dst)):
        pool.copy(a, b, rows[i] if partial else page_rows)
    pool.check()


def test_copy_of_one_page_to_many_and_onto_itself():
    pool = Pool(9, 128, 2, 64, 32)
    carat.carat_pages_copy(pool.dev[0], pool.dev[1], i32([3, 3, 3, 5]), i32([1, 2, 8, 5]),
                           **pool.scales())
    for b in (1, 2, 8):
        pool.copy(3, b, 128)
    pool.check()


def test_copy_skips_and_reports():
    pool = Pool(6, 128, 2, 64, 32)
    carat.carat_pages_copy(pool.dev[0], pool.dev[1], i32([-1, 0, -7]), i32([1, 2, 99]),
                           **pool.scales())
    pool.copy(0, 2, 128)
    pool.check()
    assert carat.carat_get_device_status(clear=True) == 0
    for src, dst, rows, bit in (([6, 1], [0, 3], [128, 5], carat.CARAT_DEV_BAD_CACHE_ID),
                                ([1, 1], [-1, 3], [1, 6], carat.CARAT_DEV_BAD_CACHE_ID),
                                ([1, 1], [4, 3], [-1, 7], carat.CARAT_DEV_BAD_CONTEXT),
                                ([1, 1], [4, 3], [129, 8], carat.CARAT_DEV_BAD_CONTEXT)):
        carat.carat_pages_copy(pool.dev[0], pool.dev[1], i32(src), i32(dst), rows=i32(rows),
                               **pool.scales())
        pool.copy(src[1], dst[1], rows[1])
        pool.check()
        assert carat.carat_get_device_status(clear=True) == bit


def test_more_jobs_than_a_grid_has_rows():
    n = 70000
    pool = Pool(100, 4, 1, 8, 0)
    src = [-1] * n
    dst = [0] * n
    for i, (a, b) in ((3, (7, 50)), (65534, (8, 51)), (65535, (9, 52)), (n - 1, (10, 53))):
        src[i], dst[i] = a, b
        pool.copy(a, b, 4)
    carat.carat_pages_copy(pool.dev[0], pool.dev[1], i32(src), i32(dst))
    pool.check()


@pytest.mark.parametrize("page_rows,kv_heads,head_dim,block_rows", SHAPES)
def test_fork(page_rows, kv_heads, head_dim, block_rows):
    max_pages, r = 5, random.Random(page_rows + head_dim)
    ctx = [0, 1, page_rows - 1, page_rows, page_rows + 1, 3 * page_rows + 17, 5 * page_rows, 200]
    pool = Pool(len(ctx) * max_pages + 20, page_rows, kv_heads, head_dim, block_rows)
    ids = r.sample(range(len(ctx) * max_pages + 20), len(ctx) * max_pages + 20)
    table = [[ids.pop() for _ in range(max_pages)] for _ in ctx]
    parents = [5, 5, 2, 0, 3, -1, 6, 4, 7, 1]
    fresh = [ids.pop() for _ in parents]
    fresh[1] = -1                                     # the parent's own last page
    fresh[6] = -5
    child = [[1000 + i] * max_pages for i in range(len(parents))]
    lengths = [-3] * len(parents)
    dchild, dlen = i32(child), i32(lengths)
    carat.carat_paged_fork(pool.dev[0], pool.dev[1], i32(table), i32(ctx), dchild, i32(parents),
                           i32(fresh), child_lengths=dlen, **pool.scales())
    for i, q in enumerate(parents):
        if q < 0:
            continue
        whole, left = divmod(ctx[q], page_rows)
        lengths[i] = ctx[q]
        child[i][:whole] = table[q][:whole]
        if whole < max_pages:
            child[i][whole] = fresh[i] if fresh[i] >= 0 else table[q][whole]
        if left and fresh[i] >= 0:
            pool.copy(table[q][whole], fresh[i], left)
    assert dchild.tolist() == child and dlen.tolist() == lengths
    pool.check()


def test_fork_skips_and_reports():
    pool = Pool(12, 128, 1, 64, 0)
    table = i32([[0, 1, 2], [3, 99, 4], [5, 6, 7]])
    for ctx, parents, fresh, bit in (
            ([10, 150, 385], [2], [8], carat.CARAT_DEV_BAD_CONTEXT),
            ([-1, 150, 10], [0], [8], carat.CARAT_DEV_BAD_CONTEXT),
            ([10, 150, 10], [3], [8], carat.CARAT_DEV_BAD_CACHE_ID),
            ([10, 150, 10], [0], [12], carat.CARAT_DEV_BAD_CACHE_ID),
            ([10, 150, 10], [1], [8], carat.CARAT_DEV_BAD_CACHE_ID)):
        child, lengths = i32([[-9, -9, -9]]), i32([-4])
        carat.carat_paged_fork(pool.dev[0], pool.dev[1], table, i32(ctx), child, i32(parents),
                               i32(fresh), child_lengths=lengths)
        assert carat.carat_get_device_status(clear=True) == bit
        assert child.tolist() == [[-9, -9, -9]] and lengths.tolist() == [-4]
    pool.check()


@pytest.mark.parametrize("page_rows,kv_heads,head_dim,block_rows", SHAPES)
@pytest.mark.parametrize("count,lines,line", [(1, 1, 1), (7, 3, 90), (20, 65, 33)])
def test_move(count, lines, line, page_rows, kv_heads, head_dim, block_rows):
    n = 2 * count + 4
    pool = Pool(n, page_rows, kv_heads, head_dim, block_rows)
    r = random.Random(count)
    ids = r.sample(range(n), n)
    src, dst = ids[:count], ids[count:2 * count]
    table = [[r.choice(ids + [-1, n, 1 << 30]) for _ in range(line)] for _ in range(lines)]
    dtable = i32(table)
    carat.carat_pages_move(pool.dev[0], pool.dev[1], i32(src + [-1]), i32(dst + [0]),
                           page_table=dtable, **pool.scales())
    to = dict(zip(src, dst))
    assert dtable.tolist() == [[to.get(e, e) for e in x] for x in table]
    for a, b in zip(src, dst):
        pool.copy(a, b, page_rows)
    pool.check()


def test_move_of_thousands_follows_in_the_table():
    n, count = 6000, 2500
    pool = Pool(n, 1, 1, 8, 0)
    ids = random.Random(1).sample(range(n), n)
    src, dst = ids[:count], ids[count:2 * count]
    table = torch.randint(0, n, (77, 501), generator=torch.Generator().manual_seed(2),
                          dtype=torch.int32)
    dtable = table.cuda()
    carat.carat_pages_move(pool.dev[0], pool.dev[1], i32(src), i32(dst), page_table=dtable)
    to = torch.arange(n, dtype=torch.int32)
    to[torch.tensor(src)] = torch.tensor(dst, dtype=torch.int32)
    assert torch.equal(dtable.cpu(), to[table.long()])
    for a, b in zip(src, dst):
        pool.copy(a, b, 1)
    pool.check()


def test_move_reports_and_leaves_the_table():
    pool = Pool(6, 128, 1, 64, 0)
    table = i32([[0, 1, 2, 5, 6, 9]])
    carat.carat_pages_move(pool.dev[0], pool.dev[1], i32([0, 9, 2]), i32([7, 1, 3]),
                           page_table=table)
    assert carat.carat_get_device_status(clear=True) == carat.CARAT_DEV_BAD_CACHE_ID
    assert table.tolist() == [[0, 1, 3, 5, 6, 9]]
    pool.copy(2, 3, 128)
    pool.check()


def test_scales_and_tables_alone():
    pool = Pool(6, 128, 2, 64, 32)
    table = i32([[0, 1], [2, 3]])
    carat.carat_pages_move(None, None, i32([2]), i32([4]), page_table=table, **pool.scales())
    for x in pool.host[2:]:
        x[4] = x[2]
    pool.check()
    assert table.tolist() == [[0, 1], [4, 3]]
    carat.carat_pages_move(None, None, i32([4]), i32([5]), page_table=table, num_pages=6)
    assert table.tolist() == [[0, 1], [5, 3]]
    pool.check()


def test_captured_lists_are_read_at_replay():
    pool = Pool(8, 128, 2, 64, 16)
    src, dst = i32([0, -1]), i32([4, 0])
    carat.carat_pages_copy(pool.dev[0], pool.dev[1], src, dst, **pool.scales())
    pool.copy(0, 4, 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        carat.carat_pages_copy(pool.dev[0], pool.dev[1], src, dst, **pool.scales())
    src.copy_(i32([1, 2]))
    dst.copy_(i32([5, 6]))
    graph.replay()
    torch.cuda.synchronize()
    pool.copy(1, 5, 128)
    pool.copy(2, 6, 128)
    pool.check()


def test_bad_arguments():
    pool = Pool(8, 128, 2, 64, 16)
    k, v, ks, vs = pool.dev
    one = i32([0])
    with pytest.raises(ValueError):
        carat.carat_pages_copy(k, v, one, i32([1, 2]), k_scales=ks, v_scales=vs)
    with pytest.raises(ValueError):
        carat.carat_pages_copy(k, v, one, one.cpu(), k_scales=ks, v_scales=vs)
    with pytest.raises(TypeError):
        carat.carat_pages_copy(k, v, one.long(), one, k_scales=ks, v_scales=vs)
    with pytest.raises(ValueError):
        carat.carat_pages_copy(k, v, one, one, k_scales=ks)
    with pytest.raises(ValueError):
        carat.carat_pages_move(k, None, one, one)
    with pytest.raises(ValueError):
        carat.carat_pages_move(None, None, one, one)
    table = i32([[0, 1]])
    with pytest.raises(carat.CaratError):             # a table forked onto itself
        carat.carat_paged_fork(k, v, table, one, table, one, one, k_scales=ks, v_scales=vs)
    carat.carat_pages_copy(k, v, one[:0], one[:0], k_scales=ks, v_scales=vs)
    carat.carat_pages_move(k, v, one[:0], one[:0], k_scales=ks, v_scales=vs)
    pool.check()
