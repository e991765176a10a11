"""Chunk attention where one workspace does not hold every sequence's operand images, and over contexts of
several hundred thousand tokens.

The reference is float64 over the values that read gives (FP8 codes are bf16 numbers, so they are the
store's); the bound is test_gpu_attend's, with fp32 sums of n terms taken as n 2^-24."""
import math

import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc

pytestmark = pytest.mark.gpu

HQ, HKV = 16, 8


def test_images_in_groups():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lens = [262145 + 37, 262144 + 500, 900]                # 2050, 2052 and 8 tiles of 8 heads, 64 KB each
    g = torch.Generator(device="cuda").manual_seed(5)
    c = wc.Cache(1, HQ, HKV, 3, max(lens), "fp8_e4m3")
    K = torch.randn(sum(lens), HKV, 128, generator=g, device="cuda").bfloat16()
    V = torch.randn(sum(lens), HKV, 128, generator=g, device="cuda").bfloat16()
    c.witcert_write_ragged(0, K, V, lens)
    del K, V
    n = [150, 131, 200]                                    # over 256 rows a KV head each
    q = (2 * torch.randn(sum(n), HQ, 128, generator=g, device="cuda")).bfloat16()
    one = [c.witcert_attend_workspace(0, [m if i == k else 0 for i, m in enumerate(n)]) for k in range(3)]
    assert one[0] + one[1] > 2 << 30 and c.witcert_attend_workspace(0, n) < one[0] + one[1]
    got = c.attend(0, q, n)
    assert c.witcert_stats()["device_errors"] == 0
    row = 0
    for i, m in enumerate(n):
        k, v = c.read(0, [lens[x] if x == i else 0 for x in range(3)])
        for j, h in ((0, 0), (m // 2, 9), (m - 1, HQ - 1)):
            seen = lens[i] - m + j + 1
            kk, vv = k[:seen, h // 2].double(), v[:seen, h // 2].double()
            x = q[row + j, h].double()
            p = torch.softmax(kk @ x / math.sqrt(128), 0)
            want = p @ vv
            d = 2.0 ** -11 * (kk.abs() @ x.abs()).max() / math.sqrt(128)
            rel = torch.exp(2 * d) * (1 + 2.0 ** -11) ** 2 - 1 + 2.0 ** -11 + seen * 2.0 ** -24
            bound = rel * (p @ vv.abs()) + 2.0 ** -8 * want.abs()
            assert ((got[row + j, h].double() - want).abs() <= bound).all()
        row += m
        del k, v
