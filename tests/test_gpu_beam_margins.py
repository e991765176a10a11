"""Selections whose scores lie near their rows' log sum exp: the sum cancels the score, and what a key's 32 bits
lost then is as large as the key.

The filter in 32 bits may pass too many candidates to the 64-bit order, never too few: every place is filled, in
order.  Tolerances are test_gpu_beam's `check`; rows of equal logits have the same sum to the bit, so there the order is
exact."""
import math

import numpy as np
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


def near(c, steps):
    """fp32 values around c: `steps` roundings of it to either side, and a quarter to either side."""
    mid = np.float32(c)
    ulps = [mid + k * np.spacing(mid) for k in range(-steps, steps + 1)]
    return torch.tensor([*ulps, *np.linspace(c - 0.26, c + 0.26, 25)], dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 8, 64])
@pytest.mark.parametrize("V", [2, 700, 32000, 128256, 131072])
def test_equal_logits(V, n, dt):
    """All of them 0: the first n tokens, at any score."""
    s = near(math.log(V), 3).view(-1, 1)
    x = torch.zeros(1, 1, V, dtype=dt, device="cuda").expand(len(s), 1, V)
    rows, tokens = check(x, s, wc.witcert_beam_select(x, s, n), n)[1:]
    m = min(n, V)
    assert (tokens[:, :m] == np.arange(m)).all() and (rows[:, :m] == np.arange(len(s))[:, None]).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V, n", [(5, 1), (700, 8), (32000, 64), (131072, 1), (131072, 64)])
def test_small_logits(V, n, dt):
    """Largest logits from 2^-24 to 1 and the row's log sum as its score."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.stack([top * (1 - torch.rand(1, V, generator=g, device="cuda") ** 2) for top in (1.0, 0.5, 0.1, 1e-3, 2.0 ** -24)])
    x = torch.cat([x, -x, x - 0.5]).to(dt)
    lse = torch.logsumexp(x.double(), -1).float()
    for d in (-0.1, -2.0 ** -20, 0.0, 2.0 ** -20, 0.1):
        check(x, lse + d, wc.witcert_beam_select(x, lse + d, n), n)


@pytest.mark.parametrize("V", [600, 131072])
@pytest.mark.parametrize("W", [5, 32])
def test_scores_a_step_apart(V, W):
    """Beams alike but for a last bit of their scores: the best beam's tokens only."""
    base = near(math.log(V), 4)
    for n in (1, W, 64):
        for k in (W - 1, 2):
            mid = base[k % len(base)]
            s = mid.expand(3, W).clone()
            s[1, k] = torch.nextafter(mid, torch.tensor(math.inf, device="cuda"))
            s[2] = torch.nextafter(mid, torch.tensor(-math.inf, device="cuda"))
            s[2, k] = mid
            x = torch.zeros(3, W, V, device="cuda")
            rows, tokens = check(x, s, wc.witcert_beam_select(x, s, n), n)[1:]
            assert (tokens == np.arange(n)).all()
            assert (rows == np.array([[0], [W + k], [2 * W + k]])).all()
