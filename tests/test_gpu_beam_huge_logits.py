"""Rows whose running maximum passes +-2^16, where the scan goes over from sums relative to the maximum's rounded
product to sums relative to the maximum itself, or back.

128 beams of ten chunks: a warp goes through five chunks of a row and raises its maximum at up to four of them, by a
little (the older part of the sum stays most of it) or by e^2.  A raise is one exponential more, off by 2^-22: four of them
2^-20.  With the other terms as they are (exponentials 2^-22, ten steps of sums 2^-20.6, the sum's last factor 2^-22, the
merge's 2^-22) that is 2.3e-6, and within what `check` allows, 2^-18 = 3.8e-6."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc

from test_gpu_beam import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


@pytest.mark.parametrize("R", [1, 3])
@pytest.mark.parametrize("middle", [65536.0, -65536.0, 65000.0, 70000.0, -70000.0])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("slope", [0.02, 1.0])
def test_maxima_around_the_border(R, middle, order, slope):
    W, V, n = 128, 5000, 128
    g = torch.Generator(device="cuda").manual_seed(int(abs(middle)))
    chunk = torch.arange(V, device="cuda") // 512
    if order == "falling":
        chunk = 9 - chunk
    elif order == "mixed":
        chunk = torch.tensor([3, 0, 8, 1, 9, 5, 2, 7, 4, 6], device="cuda")[chunk]
    # chunks' maxima from half the slope's range below the middle to half above it, and a row's share of a slope
    off = torch.rand(R, W, V, generator=g, device="cuda") * -0.4 + torch.rand(R, W, 1, generator=g, device="cuda") * slope
    x = middle + ((chunk - 5) * slope + off)
    s = 2.0 * torch.randn(R, W, generator=g, device="cuda")
    check(x, s, wc.witcert_beam_select(x, s, n), n)
