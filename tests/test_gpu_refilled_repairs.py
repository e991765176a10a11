"""Repaired blocks that are truncated away and filled with other tokens.

A block keeps its slot in the exact-key pool, so the new tokens' keys are exact as well: the decode
attends over them, their witnesses are zero, and with them the Tier A meter and the block's risk."""
import math

import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

pytestmark = pytest.mark.gpu

SCHEMES = ["int8_dither", "fp8_e4m3", "kivi2", "int8_rtn", "blackbox"]
HQ, HKV = 4, 2


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", ["bulk", "single", "rope", "ragged"])
def test_refilled_blocks_stay_exact(scheme, dtype, how):
    g = torch.Generator().manual_seed(3)
    draw = lambda n: tuple((2 * torch.randn(1, n, HKV, 128, generator=g)).to("cuda", dtype) for _ in range(2))
    hat = lambda k, v: (k * 0.875, v) if scheme == "blackbox" else ()
    c = wc.Cache(1, HQ, HKV, 1, 64, scheme, dtype=dtype, seed=6, max_repair_blocks=32)
    rope = wc.Rope(128) if how == "rope" else None
    turn = lambda k, at: k if rope is None else wc.witcert_rope(rope, at + torch.arange(k.shape[1], device="cuda"), k[0])[None]

    def append(k, v):
        h = hat(k, v)
        if rope is not None:
            c.witcert_write_rope(0, k, v, rope, *h)
        elif how == "ragged":
            c.witcert_write_ragged(0, k[0], v[0], [k.shape[1]], *(x[0] for x in h))
        elif how == "single":
            for t in range(k.shape[1]):
                part = [x[:, t:t + 1].contiguous() for x in (k, v) + h]
                (c.witcert_write_hat if h else c.witcert_write)(0, *part)
        else:
            (c.witcert_write_hat if h else c.witcert_write)(0, k, v, *h)

    q = torch.randn(1, HQ, 128, generator=g).to("cuda", dtype)
    K, V = draw(48)
    append(K, V)
    c.decode(0, q, 1e-2)
    c.witcert_gate(0, 0.0)                                 # every block's keys come back exact
    assert c.witcert_gate_stats()["blocks_paged_in"] == 3 * HKV
    c.witcert_truncate(0, [16])
    K2, V2 = draw(32)
    append(K2, V2)
    keys = torch.cat([turn(K[:, :16], 0), turn(K2, 16)], 1)
    assert torch.equal(c.read(0, [48])[0], keys[0])
    assert not c.export(0, _lib.X_WITNESS).any()
    out, m = c.decode(0, q, 1e-2)
    # the meters carry an allowance of 2^-100 (and 0 for nothing at all)
    assert (m["raw_a"] <= 2.0 ** -99).all()
    assert (c.export(0, _lib.X_BLOCK_RISK) <= 2.0 ** -99).all()
    k, v = keys[0].double(), c.read(0, [48])[1].double()
    for j in range(HQ):
        h = j // (HQ // HKV)
        p = torch.softmax(k[:, h] @ q[0, j].double() / math.sqrt(128), 0)
        assert (p @ v[:, h] - out[0, j].double()).abs().max() <= 2e-3 * v.abs().max()
