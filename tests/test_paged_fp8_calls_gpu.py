"""Calls of the attention over e4m3 pages that its schedule treats apart: more
requests than the range search keeps counts of, one long request among short ones;
and refusals of numbers that do not fit an int (GPU, against 64 bits)."""
import pytest
import torch

from sliding_window_gqa_ring_gb300 import carat
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
