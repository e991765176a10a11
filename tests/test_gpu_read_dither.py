"""Reads of the dithered store take the whole dither off.

A zero in a group with a larger element has code 0, so it stands for -s xi: xi has 24 bits, -xi is an
fp32 number, and only the product with s is rounded (fp32: half a step of it, 2^-24), then the output."""
import numpy as np
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from oracle.philox import dither

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [40, 700])                    # blocks by quarters of a warp's work, and whole ones
def test_zeros_stand_for_the_dither(dtype, n):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hkv, seed, offset = 96, 77, 9
    x = torch.zeros(1, n, hkv, 128)
    x[..., ::32] = 127.0 * 2.0 ** -3                        # s = 2^-3 exactly
    c = wc.Cache(1, hkv, hkv, 1, n, "int8_dither", dtype=dtype, seed=seed, pos_offset=offset)
    c.witcert_write(0, x.to("cuda", dtype), x.to("cuda", dtype))
    half = torch.finfo(dtype).eps / 2
    other = np.arange(128) % 32 != 0
    for tensor, got in enumerate(c.read(0, [n])):
        got = got.double().cpu().numpy()
        for h in range(0, hkv, 5):
            want = -(2.0 ** -3) * dither(seed, 0, h, np.arange(offset, offset + n), tensor).astype(np.float64)
            err = np.abs(got[:, h] - want)[:, other]
            assert np.all(err <= half * np.abs(want[:, other]))      # s is a power of two: one rounding
