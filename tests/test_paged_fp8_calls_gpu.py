"""Windows of the attention over e4m3 pages that do not fit an int (GPU)."""
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
