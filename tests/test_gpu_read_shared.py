"""Reads of several sequences of the dithered store at once, which share the dither of a place, give what reads of
each sequence alone give, to the bit."""
import random

import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


def alone(c, n, t0):
    B = len(n)
    parts = [c.read(0, [n[i] if k == i else 0 for k in range(B)], t0) for i in range(B)]
    return [torch.cat(x) for x in zip(*parts)]


@pytest.mark.parametrize("kind", ["contiguous", "paged", "fp32", "repaired", "offset"])
@pytest.mark.parametrize("lens", [[40] * 2, [700, 690, 701, 3], [0, 2000, 17, 1999, 2000], [33] * 150, [5000] * 3 + [16]])
def test_together_and_alone(kind, lens):
    r, B = random.Random(len(lens) + lens[0]), len(lens)
    torch.manual_seed(B)
    dtype = torch.float32 if kind == "fp32" else torch.bfloat16
    kw = dict(max_pages=sum((x + 15) // 16 for x in lens)) if kind == "paged" else {}
    if kind == "repaired":
        kw["max_repair_blocks"] = 4096
    c = wc.Cache(1, 4, 2, B, max(lens), "int8_dither", dtype=dtype, seed=5, pos_offset=1000 * (kind == "offset"), **kw)
    k = 3 * torch.randn(sum(lens), 2, 128, device="cuda").to(dtype)
    c.witcert_write_ragged(0, k, k, lens)
    if kind == "repaired":
        c.decode(0, torch.randn(B, 4, 128, device="cuda").to(dtype), 1e-2)
        c.witcert_gate(0, 1e-4)
        assert c.witcert_gate_stats()["blocks_paged_in"] > 0
    for n in (lens, [min(x, 30) for x in lens], [r.randint(0, x) for x in lens], [x // 2 for x in lens]):
        for t0 in (None, [r.randint(0, x - m) for x, m in zip(lens, n)], [0] * B):
            for a, b in zip(c.read(0, n, t0), alone(c, n, t0)):
                assert torch.equal(a, b)
