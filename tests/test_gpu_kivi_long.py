"""A two-bit append of more blocks than a grid's second dimension holds stores what shorter ones do."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("turn", [False, True])
def test_blocks_beyond_65535(turn):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n = 16 * 65535 + 16 * 70 + 5
    g = torch.Generator(device="cuda").manual_seed(2)
    K, V = (torch.randn(1, n + 3, 1, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    rope = wc.Rope(128, base=1e6)
    whole, parts = (wc.Cache(1, 1, 1, 1, n + 3, "kivi2") for _ in range(2))

    def write(c, a, b):
        part = K[:, a:b].contiguous(), V[:, a:b].contiguous()
        if turn:
            c.witcert_write_rope(0, *part, rope)
        else:
            c.witcert_write(0, *part)

    write(whole, 0, 3)                                     # the first finished block starts in the tail
    write(whole, 3, n + 3)
    for a in range(0, n + 3, 300000):
        write(parts, a, min(a + 300000, n + 3))
    for a, b in zip(whole.read(0, [n + 3]), parts.read(0, [n + 3])):
        assert torch.equal(a, b)
    for kind in (_lib.X_K_CODES, _lib.X_V_CODES, _lib.X_KIVI_K_SCALE, _lib.X_WITNESS):
        a, b = whole.export(0, kind), parts.export(0, kind)
        m = (n + 3) // 16 * (1 if kind == _lib.X_KIVI_K_SCALE else 16)
        assert torch.equal(a[:, :m].view(torch.uint8), b[:, :m].view(torch.uint8))
