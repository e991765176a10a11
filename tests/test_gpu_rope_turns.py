"""Turns per position: frequencies of either sign and of any size, at far positions.

The bound is test_gpu_rope's: half a step of the output, 16 units of 2^-24 (|a| + |b|) of fp32 evaluation
and the frequency's own rounding; plus the turn's step of 2^-64, position x 2^-65 turns."""
import math

import numpy as np
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc

from test_gpu_rope import want_rotation

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


def check(rope, pos, seed):
    q = torch.randn(len(pos), 2, 128, generator=torch.Generator().manual_seed(seed)).cuda()
    got = wc.witcert_rope(rope, pos.cuda(), q)
    want, slack = want_rotation(q, pos, rope)
    r = rope.rotary_dim
    mag = q.abs().double().cpu().numpy()
    mag = mag[..., :r].reshape(len(pos), 2, 2, r // 2).sum(2) * abs(rope.scale)      # |a| + |b| of a pair
    step = 2 * math.pi * np.abs(pos.double().numpy())[:, None, None] * 2.0 ** -65 * mag
    slack[..., :r] += np.concatenate([step, step], -1)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= slack + 2.0 ** -24 * (np.abs(want) + slack)), float((err / (slack + 2.0 ** -24 * np.abs(want))).max())


def test_small_frequencies_of_either_sign():
    base = [1e-3 * 10 ** (-p / 4) for p in range(64)]       # 1e-3 .. 1.8e-19
    pos = torch.tensor([1, -1, 4097, 2 ** 31 + 5, -2 ** 36 - 7, 2 ** 40 + 3])
    for sign in (1, -1):
        check(wc.Rope(128, freq=[sign * f for f in base]), pos, 4)


def test_large_frequencies_of_either_sign():
    freq = [(-1) ** p * 1.37 ** p for p in range(32)]       # up to 1.7e4 radians a position
    check(wc.Rope(64, freq=freq), torch.tensor([0, 1, -3, 70001, 2 ** 20 + 1]), 5)


def test_slow_pairs_far_out():
    check(wc.Rope(128, base=5e6), torch.tensor([2 ** 30 + 1, 2 ** 36 - 5, -2 ** 38 + 9]), 6)


def test_a_frequency_and_its_negative_turn_opposite_ways():
    f = [0.3 / (p + 1) for p in range(64)]
    pos = torch.tensor([5, 1000, 2 ** 33 + 1])
    q = torch.randn(3, 2, 128, generator=torch.Generator().manual_seed(7)).cuda()
    a = wc.witcert_rope(wc.Rope(128, freq=f), pos.cuda(), q, inverse=True)
    b = wc.witcert_rope(wc.Rope(128, freq=[-x for x in f]), pos.cuda(), q)
    assert torch.equal(a, b)
