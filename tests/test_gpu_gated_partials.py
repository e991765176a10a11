"""A context-parallel shard's record from a cache with the gate enabled.

The record, merged alone, is the decode of that cache: same kernels, same splits, so the same bits; and
the block risks of the last whole decode stay as they were, for witcert_gate."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

pytestmark = pytest.mark.gpu

HQ, HKV = 6, 2


@pytest.mark.parametrize("scheme", ["int8_dither", "fp8_e4m3", "kivi2", "int8_rtn", "blackbox"])
@pytest.mark.parametrize("pages", [0, 80])
@pytest.mark.parametrize("v_witness", [False, True])
def test_partial_records_of_a_gated_cache(scheme, pages, v_witness):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator().manual_seed(4)
    K, V = (torch.randn(2, 300, HKV, 128, generator=g).bfloat16().cuda() for _ in range(2))
    c = wc.Cache(1, HQ, HKV, 2, 320, scheme, seed=5, max_repair_blocks=16, max_pages=pages, v_witness=v_witness)
    if scheme == "blackbox":
        c.witcert_write_hat(0, K, V, K * 0.9375, V * 0.9375)
    else:
        c.witcert_write(0, K, V)
    q, q2 = (torch.randn(2, HQ, 128, generator=g).bfloat16().cuda() for _ in range(2))
    for repaired in (False, True):
        out, m = c.decode(0, q, 1e-2)
        risk = c.export(0, _lib.X_BLOCK_RISK)
        for query, want in ((q, (out, m)), (q2, None)):
            rec = c.decode_partial(0, query, 1e-2, 300)
            got, gm = wc.witcert_merge_partials(rec[:, :, None].contiguous(), scheme)
            if want is not None:
                # the record's sums are merged once more, each rounded once: a few units of 2^-24
                assert (got - out).abs().max() <= 2.0 ** -20 * out.abs().max()
                assert ((gm["raw_a"] - m["raw_a"]).abs() <= 2.0 ** -19 * m["raw_a"] + 2.0 ** -99).all()
        assert torch.equal(c.export(0, _lib.X_BLOCK_RISK).view(torch.int32), risk.view(torch.int32))
        if not repaired:
            c.witcert_gate(0, 0.0)                         # some blocks are exact in the second round
            assert c.witcert_gate_stats()["blocks_paged_in"] == 16
